// k_ffn_gated.cu -- the ring's kernels of the gated product, and the planner of all products.
#include <initializer_list>
#include "ffn_ring.cuh"

namespace gp {

cudaError_t launch_ffn_gated(FfnProduct& p, const void** kernel) { return launch_tile<true, false, false>(p, kernel); }

namespace {

// Pairs that fit on the device at once (cached per device).
cudaError_t pair_capacity(int* pairs) {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && (*pairs = cached[dev].load()) > 0) return cudaSuccess;
  using Sh = RingShape<256, true, kCodes>;
  const void* k = reinterpret_cast<const void*>(ffn_ring_kernel<256, true, kCodes, true, false, false>);
  if ((e = ensure_smem_attr(k, Sh::SMEM)) != cudaSuccess) return e;
  RingConfig c(2, Sh::THREADS, 2, Sh::SMEM, nullptr);
  if ((e = cudaOccupancyMaxActiveClusters(pairs, k, &c.cfg)) != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorLaunchOutOfResources;
  if (dev >= 0 && dev < 64) cached[dev].store(*pairs);
  return cudaSuccess;
}

template <int BN, bool PAIR, RingOut OUT>
void ring_shape_of(gp_plan* p) {
  using Sh = RingShape<BN, PAIR, OUT>;
  p->stages = Sh::STAGES;
  p->stage_bytes = Sh::STAGE;
  p->ring_bytes = Sh::STAGES * Sh::STAGE;
  p->smem_bytes = Sh::SMEM;
  p->tmem_cols = Sh::TMEM_COLS;
  p->threads = Sh::THREADS;
}

int64_t blocks(int64_t n, int64_t of) { return (n + of - 1) / of; }

// The tiles of pairs behind the last full round are cut in halves where those make one round at most (not where a group
// of 128 columns kept in 8 bits would be cut: whole_groups).
void ffn_cut_tail(gp_plan* p, bool whole_groups) {
  const int64_t pairs = p->grid / 2, rest = p->cta_pair && pairs > 0 ? p->tiles % pairs : 0;
  p->half_tiles = !whole_groups && p->tiles > pairs && 2 * rest <= pairs ? static_cast<int32_t>(rest) : 0;
  p->dp_tiles = static_cast<int32_t>(p->tiles) - p->half_tiles;
}

}  // namespace

int ffn_plan_impl(int op, int64_t rows, int64_t cols, int64_t summed, int count, bool wide_sums, bool codes, bool bf16, int sms,
                  const gp_ffn_options* opts, gp_plan* p) {
  std::memset(p, 0, sizeof(*p));
  const int want = opts ? opts->tile : 0;
  constexpr int kSplit128 = 129;   // 128 x 128 by a cluster; 128: by the ring
  bool known = false;
  for (int t : {0, 16, 32, 64, 128, kSplit128, 256}) known |= want == t;
  if (!known) return GP_ERR_UNSUPPORTED;
  const bool gated = op == kFfnGated;
  const bool lose = opts && opts->inject_lost_load;
  const int have = sms > 0 ? sms : 152;
  const bool can_pair = have >= 2 && !lose, can_one = !(gated && codes), can_few = !codes;
  const int64_t kt = blocks(summed, kFfnBK) * (op == kFfnInputGrad ? count : 1);
  const int64_t problems = op == kFfnWeightGrad ? count : 1;
  auto few_tiles = [&](int bn) { return problems * blocks(cols, 128) * blocks(rows, bn); };
  const int want_splits = opts ? opts->k_splits : 0;
  if (want_splits != 0 && want_splits != 1 && want_splits != 2 && want_splits != 4 && want_splits != 8) return GP_ERR_UNSUPPORTED;
  // CTAs that share a tile's K blocks: as many as the SMs take at once (16 clusters of 8 do not fit on 152: 128 rows of a
  // weight gradient by 8 CTAs 20.7 us, by 4 13.3), with four K blocks each at least
  auto few_ctas = [&](int bn) {
    if (want_splits) return want_splits;
    int c = 1;
    while (c < ffn_few_most_ctas(bn) && few_tiles(bn) * c * 2 <= (c == 4 ? have * 3 / 4 : have) && kt >= 4 * c * 2) c *= 2;
    return c;
  };
  int tile = want;
  if (tile == 0) {
    // The least estimate, in ns, as measured on a 152-SM GB300 (device time of calls in a graph): a call with one K
    // block, each further one on the busiest SM, and each further round of tiles; but not less than the operands take
    // from HBM.  For example 1000 x 776 x 2048: 64 rows 10.5 us, 128 rows by two CTAs 11.0, 128 x 128 13; 512 x 4096 x
    // 4096: 128 x 128 20.6, 128 rows 22.1, 256 x 256 29; gated 333 x 1000 x 776: 128 x 128 8.7, 256 x 256 10.0, 64 rows by
    // two CTAs 10.0; weight gradient of 8192 x 512 x 512: 64 rows by four CTAs 10.5, by one 21.1, 128 x 128 26.4.
    const double read = 2.0 * (static_cast<double>(rows) * summed + (gated ? 2.0 : 1.0) * cols * summed) * (kt > 0 ? count : 0) / 6500;
    // Boxes whose rows begin off 128-byte boundaries take longer to load.  The planner does not see pointers and row
    // strides: it takes rows to be packed, so that K says where they begin.  Rows of 2056 values laid out 2112 apart are
    // counted as slow without reason, rows of 2048 laid out 2056 apart as fast; the gradients' are counted as fast.
    const double slow = (op == kFfnLinear || gated) && summed % 64 ? 1.6 : 1.0;
    double best = 0;
    auto take = [&](int t, double once, double k_blocks) {
      const double ns = once + (k_blocks > read ? k_blocks : read);
      if (tile == 0 || ns < best) {
        tile = t;
        best = ns;
      }
    };
    if (can_few) {
      constexpr int kRows[4] = {16, 32, 64, 128}, kBlock[2][4] = {{130, 110, 150, 220}, {217, 230, 265, 0}};
      for (int i = op == kFfnWeightGrad ? 2 : 0; i < (gated ? 3 : 4); ++i) {
        const int bn = kRows[i], c = few_ctas(bn);
        if (c > ffn_few_most_ctas(bn)) continue;
        const double rounds = static_cast<double>(blocks(few_tiles(bn) * c, have));
        const double again = (blocks(rows, bn) - 1) * (bn < 64 ? 1500 : 0);   // the other operand once more from L2
        const double once = 4500 + bn * 15 + (gated ? 2000 : 0) + (c > 1 ? 700 : 0) + again;
        take(bn == 128 ? kSplit128 : bn, once + (rounds - 1) * once, rounds * blocks(kt, c) * kBlock[gated][i] * slow);
      }
    }
    const int64_t pairs = problems * blocks(rows, 256) * blocks(cols, gated ? 128 : 256);
    const int64_t ones = problems * blocks(rows, 128) * blocks(cols, gated ? 64 : 128);
    const double one_rounds = static_cast<double>(blocks(ones, have)), pair_rounds = static_cast<double>(blocks(pairs, have / 2 > 0 ? have / 2 : 1));
    // (few rows leave most of an operand's slot empty, and the loads under way are too few: gated 1 x 8192 x 4096 36.6 us
    // by 128 x 128, 22.6 by 16 rows)
    const bool whole = rows > 64 || !can_few;
    if (can_one && whole) take(128, 5500 + (one_rounds - 1) * 800, one_rounds * kt * 210 * slow);
    if (can_pair && (whole || !can_one)) take(256, 6500 + (pair_rounds - 1) * 1500, pair_rounds * kt * 285 * slow);
    if (tile == 0) return GP_ERR_UNSUPPORTED;   // (kept in 8 bits on one SM: a pair of CTAs does not fit)
  }
  const bool few = tile < 128 || tile == kSplit128;
  if ((tile == 256 && !can_pair) || (tile == 128 && !can_one) || (few && !can_few) || (tile < 64 && op == kFfnWeightGrad) ||
      (tile == kSplit128 && gated))
    return GP_ERR_UNSUPPORTED;
  p->dtype = GP_PLAN_FFN;
  p->variant = GP_PIPELINED;
  p->bk = kFfnBK;
  p->k_tiles = kt;
  p->k_splits = 1;
  // Row blocks that are walked together, so that the columns' weights come from L2. In short runs / kept up, us:
  // linear 8192 x 8192 x 4096 8: 280 / 316, 12: 277 / 312, 16: 274 / 309, 32: 288 / 336; gated 4096 x 8192 x 4096
  // into 8 bits 293 / 328, 294 / 328, 288 / 320, 288 / 318; linear 4096 x 8192 x 8192 287 / 319 against 289 / 324
  // with 16. The gradients of 2 x 4096 x 8192 x 4096: to the input 341 / 370 against 346 / 375, to the weights the
  // same, 348 / 384 with 32.
  p->raster_gm = (op == kFfnLinear || op == kFfnGated) ? 16 : 8;
  if (few) {
    if (tile == kSplit128) tile = 128;
    p->kernel = gated ? "ffn_few_gated" : "ffn_few";
    p->layout = 1;
    p->bm = 128;
    p->bn = tile;
    ffn_few_shape(p, tile, gated);
    p->tiles = few_tiles(tile);
    const int c = few_ctas(tile);
    if (c > ffn_few_most_ctas(tile)) return GP_ERR_UNSUPPORTED;
    p->k_splits = c;
    if (p->tiles > kFfnMaxTiles / 8) return GP_ERR_SIZE;
    p->grid = sms > 0 ? static_cast<int32_t>(p->tiles * c) : 0;
  } else {
    p->kernel = tile == 256 ? "ffn_pair_ring" : "ffn_ring";
    p->persistent = 1;
    p->cta_pair = tile == 256;
    p->bm = tile;
    p->bn = gated ? tile / 2 : tile;
    const bool hold = wide_sums || kt > ffn_restart(false, bf16);
    if (tile == 256)
      hold ? ring_shape_of<256, true, kHold>(p) : ring_shape_of<256, true, kStream>(p);
    else
      hold ? ring_shape_of<128, false, kHold>(p) : ring_shape_of<128, false, kStream>(p);
    const int64_t r = blocks(rows, p->bm), c = blocks(cols, p->bn);
    if (r > kFfnMaxTiles / c / problems) return GP_ERR_SIZE;
    p->tiles = r * c * problems;
    const int64_t ctas = p->cta_pair ? 2 : 1, workers = sms / ctas;
    p->grid = static_cast<int32_t>(ctas * (p->tiles < workers ? p->tiles : workers));
  }
  ffn_cut_tail(p, gated && codes);
  p->compute_load_ratio = 2.0 * p->bm * p->bn / (p->bm + p->bn);
  return GP_OK;
}

cudaError_t ffn_fit_pairs(gp_plan* plan, bool whole_groups) {
  if (!plan->cta_pair) return cudaSuccess;
  int pairs = 0;
  const cudaError_t e = pair_capacity(&pairs);
  if (e == cudaSuccess && 2 * pairs < plan->grid) {
    plan->grid = 2 * pairs;
    ffn_cut_tail(plan, whole_groups);
  }
  return e;
}

}  // namespace gp
