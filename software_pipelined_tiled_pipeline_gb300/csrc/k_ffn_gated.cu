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
  using Sh = RingShape<256, true, kHold>;
  const void* k = reinterpret_cast<const void*>(ffn_ring_kernel<256, true, kHold, true, false, false>);
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

}  // namespace

int ffn_plan_impl(int op, int64_t rows, int64_t cols, int64_t summed, int count, bool wide_sums, bool codes, int sms,
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
  // CTAs that share a tile's K blocks: as many as the SMs take at once, with four K blocks each at least
  auto few_ctas = [&](int bn) {
    if (want_splits) return want_splits;
    int c = 1;
    while (c < ffn_few_most_ctas(bn) && few_tiles(bn) * c * 2 <= have && kt >= 4 * c * 2) c *= 2;
    return c;
  };
  int tile = want;
  if (tile == 0) {
    // Estimates in ns: K blocks one after another on the busiest SM, and the rest of a call.
    double best = 0;
    auto take = [&](int t, double ns) {
      if (tile == 0 || ns < best) {
        tile = t;
        best = ns;
      }
    };
    if (can_few) {
      for (int bn = op == kFfnWeightGrad ? 64 : 16; bn <= (gated ? 64 : 128); bn *= 2) {
        const int64_t t = few_tiles(bn);
        const int c = few_ctas(bn);
        take(bn == 128 ? kSplit128 : bn, static_cast<double>(blocks(t * c, have)) * (blocks(kt, c) * (gated ? 300 : 200) + 2500 + bn * 25) + (c > 1 ? 1500 : 0));
      }
    }
    const int64_t pairs = problems * blocks(rows, 256) * blocks(cols, gated ? 128 : 256);
    const int64_t ones = problems * blocks(rows, 128) * blocks(cols, gated ? 64 : 128);
    if (can_one) take(128, static_cast<double>(blocks(ones, have)) * kt * 260 + 6000);
    if (can_pair) take(256, static_cast<double>(blocks(pairs, have / 2)) * kt * 280 + 8000);
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
  p->raster_gm = 8;
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
    const bool hold = wide_sums;
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
  p->dp_tiles = static_cast<int32_t>(p->tiles);
  p->compute_load_ratio = 2.0 * p->bm * p->bn / (p->bm + p->bn);
  return GP_OK;
}

cudaError_t ffn_fit_pairs(gp_plan* plan) {
  if (!plan->cta_pair) return cudaSuccess;
  int pairs = 0;
  const cudaError_t e = pair_capacity(&pairs);
  if (e == cudaSuccess && 2 * pairs < plan->grid) plan->grid = 2 * pairs;
  return e;
}

}  // namespace gp
