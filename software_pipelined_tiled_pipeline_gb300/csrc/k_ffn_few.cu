// k_ffn_few.cu -- the products of small problems: for few tokens, and where the
// ring's tiles would leave SMs idle.  The operand whose rows are the output's
// columns (a weight, or x in a weight's gradient) fills the tensor cores' M side,
// 128 rows per CTA, the other one their N side (16, 32, 64 or 128 rows; gated up to
// 64, a weight's gradient from 64), and a cluster of 1 to 8 CTAs shares a tile's K
// blocks.
//
//   s[c][r] = sum over k of p[c][k] * q[r][k];  then as in ffn_ring.cuh
//
// The sums of a cluster meet in distributed shared memory: each CTA is handed its
// share of q's rows by all, adds them in K order and writes them, neighbouring
// lanes along a row of the output.
// What bounds it: for few tokens the weight's bytes (1 x 8192 x 4096 twice, gated:
// 134 MB in 17.8 us from the first load to the last), and for one token and a
// small weight the launch, the first loads and the exchange: 3.5 of 9 us.
#include "ffn_ring.cuh"

namespace gp {
namespace {

constexpr int kFewThreads = 384;
constexpr int kFewAddThreads = 256;      // eight warps: 32 rows of the weight x half of the tokens each
constexpr int kFewMaxRing = 12;

struct FewBarriers {
  uint64_t full[kFewMaxRing];
  uint64_t empty[kFewMaxRing];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  CtaCtl ctl;
};
constexpr int kFewBarrierBytes = 256;
static_assert(sizeof(FewBarriers) <= kFewBarrierBytes, "barrier region too small");

constexpr int kFewRow = 128 + 4;         // floats of a row of the exchange: rows begin on other banks

template <int BN, bool GATED>
struct FewShape {
  static constexpr int PARTS = GATED ? 2 : 1;
  static constexpr int P_BYTES = 128 * kFfnBK * 2;
  static constexpr int STAGE = PARTS * P_BYTES + BN * kFfnBK * 2;
  static constexpr int FIXED = kFewBarrierBytes + kSmemAlignSlack;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kFewMaxRing ? FIT : kFewMaxRing;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static constexpr uint32_t TMEM_COLS = 2 * PARTS * BN;
  static constexpr int HALF = BN / 2;
  // The exchange: for each CTA of the cluster its sums of the rows of q that are this one's share, kFewRow floats each.
  static_assert(PARTS * BN * kFewRow * 4 <= STAGES * STAGE, "the exchange takes the ring's memory");
  static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS >= 32 && TMEM_COLS <= 512, "TMEM columns");
};

struct FewParams {
  FfnOut o;
  int32_t rows, cols;        // of the output
  int32_t kt;                // K blocks of one source
  int32_t sources, problems;
  int32_t restart;
  int32_t k_log;             // log2 of the CTAs that share a tile's K blocks
  int32_t row_blocks, per_problem;
  uint32_t idesc;
  KernelCtl ctl;
};

struct FewMaps {
  CUtensorMap q[2], p[2];
  CUtensorMap q64[2], p64[2];   // in boxes of 64 of their rows: an MN-major operand's end
};

__device__ __forceinline__ void tmem_ld_few(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void st_shared_f1(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f1(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_int(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// Eight neighbouring values of a row in 16 bits or FP32, `n` of which exist (8 or less).
template <typename T>
__device__ __forceinline__ void load_eight(T (&t)[8], const T* p, int n, bool vec) {
  if (vec && n >= 8) {
    uint4 w[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    memcpy(t, w, sizeof(t));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    from_f32(0.f, t[i]);
    if (i < n) t[i] = p[i];
  }
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8], int n, bool vec) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) from_f32(v[i], t[i]);
  if (vec && n >= 8) {
    uint4 w[sizeof(T) / 2];
    memcpy(w, t, sizeof(t));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = t[i];
}

__device__ __forceinline__ void add_eight(float (&v)[8], const float* from) {
  const float4 x = reinterpret_cast<const float4*>(from)[0], y = reinterpret_cast<const float4*>(from)[1];
  v[0] += x.x;
  v[1] += x.y;
  v[2] += x.z;
  v[3] += x.w;
  v[4] += y.x;
  v[5] += y.y;
  v[6] += y.z;
  v[7] += y.w;
}

// The `per` output rows from row0 on, 128 columns from col0 on, of the exchanged sums of `ctas` CTAs: sixteen threads to a
// row, eight columns each.
template <int BN, bool GATED, typename T, typename O>
__device__ __forceinline__ void finish_few(const FewParams& g, int problem, const float* buf, int t, int ctas, int per,
                                           int64_t row0, int64_t col0) {
  const FfnOut& o = g.o;
  const O* const add = static_cast<const O*>(o.add[problem]);
  O* const out = static_cast<O*>(o.out[problem]);
  T* const keep0 = static_cast<T*>(o.keep[0]);
  T* const keep1 = static_cast<T*>(o.keep[1]);
  const int lane = t & 15;
  const int64_t c = col0 + 8 * lane;
  const int n = g.cols - c < 8 ? static_cast<int>(g.cols - c) : 8;
  if (n <= 0) return;
  const bool vec = o.vec != 0;
  float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (!GATED && o.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) bias[i] = o.bias_f32 ? static_cast<const float*>(o.bias)[c + i] : to_f32(static_cast<const T*>(o.bias)[c + i]);
  }
  const int64_t left = g.rows - row0;
  const int rows = left < per ? static_cast<int>(left) : per;      // (may be < 0)
  constexpr int STEP = kFewAddThreads / 16;
  const float* const mine = buf + 8 * lane;
  // Short code, run a few times: an instruction that runs once costs more to fetch than the loop does (four rows
  // unrolled: 1000 x 776 x 2056 15.5 us).  The next row's addend is under way meanwhile.
  O was[8];
  const int i0 = t >> 4;
  if (!GATED && add && i0 < rows) load_eight(was, add + (row0 + i0) * o.ld_add[problem] + c, n, vec);
#pragma unroll 1
  for (int i = i0; i < rows; i += STEP) {
    O next[8];
    if (!GATED && add && i + STEP < rows) load_eight(next, add + (row0 + i + STEP) * o.ld_add[problem] + c, n, vec);
    float v[8], u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = 0.f;
      u[k] = 0.f;
    }
#pragma unroll 1
    for (int s = 0; s < ctas; ++s) {   // in K order
      add_eight(v, mine + (s * per + i) * kFewRow);
      if (GATED) add_eight(u, mine + (BN + s * per + i) * kFewRow);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += bias[k];
    if (keep0) {
      store_eight(keep0 + (row0 + i) * o.ld_keep[0] + c, v, n, vec);
      if (GATED) store_eight(keep1 + (row0 + i) * o.ld_keep[1] + c, u, n, vec);
    }
    activate_all(v, o.act);
    if (GATED) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= u[k];
    } else if (add) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] += to_f32(was[k]);
        was[k] = next[k];
      }
    }
    store_eight(out + (row0 + i) * o.ld_out[problem] + c, v, n, vec);
  }
}

// P_MN, Q_MN: the operand is stored summed axis first.
template <int BN, bool GATED, bool P_MN, bool Q_MN>
__global__ void __launch_bounds__(kFewThreads, 1)
    ffn_few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewParams g) {
  using Sh = FewShape<BN, GATED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewBarriers* bar = reinterpret_cast<FewBarriers*>(ring + Sh::STAGES * Sh::STAGE);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int ctas = 1 << g.k_log;
  const uint32_t rank = ctas > 1 ? cluster_ctarank() : 0u;
  const int tile = static_cast<int>(blockIdx.x) >> g.k_log;
  // row blocks of one column block side by side: p's rows are read from L2 after the first
  const int problem = tile >= g.per_problem ? 1 : 0, in = tile - problem * g.per_problem;
  const int pb = in / g.row_blocks, qb = in - pb * g.row_blocks;
  const int kt = g.kt * g.sources;
  const int k0 = static_cast<int>((static_cast<int64_t>(kt) * rank) >> g.k_log);
  const int k1 = static_cast<int>((static_cast<int64_t>(kt) * (rank + 1)) >> g.k_log);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Sh::STAGES; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->acc_full[a], 1);
      mbar_init(&bar->acc_empty[a], kFewAddThreads / 32);
    }
    mbar_init(&bar->drain, 1);
    bar->ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, Sh::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  // While the work before this kernel finishes, its first boxes come into L2:
  // a prefetch writes nothing, and L2 stays coherent with what is still written.
  if (!P_MN && warp == 0 && lane == 0) {
    for (int kb = k0; kb < k1 && kb < k0 + Sh::STAGES; ++kb) {
      tma_prefetch_l2_2d(&maps.p[0], kb * kFfnBK, pb * 128);
      if (GATED) tma_prefetch_l2_2d(&maps.p[1], kb * kFfnBK, pb * 128);
      tma_prefetch_l2_2d(&maps.q[0], kb * kFfnBK, qb * BN);
    }
  }
  pdl_wait();
  const uint32_t tmem = bar->tmem_base;
  CtaCtl* cta = &bar->ctl;
  RingProducer prod(warp);

  if (warp < 4) {
    if (warp != 1 && lane == 0) {
      // ---------------- producers ----------------
      const bool lose = g.ctl.inject_lost_load && tile == static_cast<int>(gridDim.x >> g.k_log) - 1;
      const int p_boxes = P_MN ? mn_boxes(pb * 128, g.cols) : 0, q_boxes = Q_MN && BN == 128 ? mn_boxes(qb * BN, g.rows) : 0;
      const uint32_t bytes = Sh::STAGE - (p_boxes == 1 ? 8192 : 0) - (q_boxes == 1 ? 8192 : 0);
      for (int kb = k0 + prod.which; kb < k1; kb += kRingProducers) {
        const int s = prod.slot;
        if (!mbar_wait(&bar->empty[s], prod.phase ^ 1u, g.ctl, cta, kSiteProducerEmpty) || cta->abort) break;
        const uint32_t at = smem_u32(ring + s * Sh::STAGE);
        if (lose && kb == kt - 1) {   // test hook: this load never comes
          prod.lost = prod.issued;
        } else {
          const int second = kb >= g.kt ? 1 : 0, k = (kb - second * g.kt) * kFfnBK;
          const CUtensorMap* mp = &maps.p[second];
          const CUtensorMap* mq = &maps.q[problem | second];
          mbar_arrive_expect_tx(&bar->full[s], bytes);
          if (!P_MN) {
            tma_load_2d(at, mp, &bar->full[s], k, pb * 128);
            if (GATED) tma_load_2d(at + Sh::P_BYTES, &maps.p[1], &bar->full[s], k, pb * 128);
          } else if (p_boxes == 0) {
            tma_load_3d(at, mp, &bar->full[s], 0, k, pb * 2);
          } else {
            tma_load_2d(at, &maps.p64[second], &bar->full[s], pb * 128, k);
            if (p_boxes == 2) tma_load_2d(at + 8192, &maps.p64[second], &bar->full[s], pb * 128 + 64, k);
          }
          const uint32_t q_at = at + Sh::PARTS * Sh::P_BYTES;
          if (!Q_MN) {
            tma_load_2d(q_at, mq, &bar->full[s], k, qb * BN);
          } else if (BN == 128 && q_boxes == 0) {
            tma_load_3d(q_at, mq, &bar->full[s], 0, k, qb * 2);
          } else {
            tma_load_2d(q_at, &maps.q64[problem | second], &bar->full[s], qb * BN, k);
            if (BN == 128 && q_boxes == 2) tma_load_2d(q_at + 8192, &maps.q64[problem | second], &bar->full[s], qb * BN + 64, k);
          }
        }
        prod.advance(Sh::STAGES);
      }
    } else if (warp == 1 && ring_elect_one()) {
      // ---------------- MMA issuer (one lane) ----------------
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      const uint32_t ring0 = smem_u32(ring);
      const uint64_t p0 = P_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0);
      const uint64_t q0 = (Q_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0)) + Sh::PARTS * Sh::P_BYTES / 16;
      constexpr uint32_t P_STEP = P_MN ? 128 : 2, Q_STEP = Q_MN ? 128 : 2;   // 16 along K, as in the ring
      for (int kc = k0; ok && kc < k1; kc += g.restart) {
        const int end = min(kc + g.restart, k1);
        if (!mbar_wait(&bar->acc_empty[a], aph ^ 1u, g.ctl, cta, kSiteMmaAccEmpty)) break;
        tc_fence_after();
        const uint32_t d = tmem + a * Sh::PARTS * BN;
        for (int kb = kc; kb < end; ++kb) {
          // (nothing is issued of a slot that never came)
          if (!mbar_wait(&bar->full[s], ph, g.ctl, cta, kSiteConsumerFull)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dp = p0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
          const uint64_t dq = q0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
#pragma unroll
          for (int kk = 0; kk < kFfnBK / 16; ++kk) {
            const uint32_t more = kb > kc || kk > 0;
            umma_f16(d, dp + P_STEP * kk, dq + Q_STEP * kk, g.idesc, more);
            if (GATED) umma_f16(d + BN, dp + Sh::P_BYTES / 16 + P_STEP * kk, dq + Q_STEP * kk, g.idesc, more);
          }
          umma_commit(&bar->empty[s]);
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&bar->acc_full[a]);
        if (++a == 2) { a = 0; aph ^= 1u; }
      }
      // fires when every MMA issued above has completed
      umma_commit(&bar->drain);
      CtaCtl never_abort{0};
      mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
    }
    __syncwarp();
    if (ctas > 1) {
      // the writing warps' two barriers around their exchange (below); between
      // them a CTA that gave up tells the others, so that none of them writes
      // what its sums are missing from
      cluster_sync();
      if (warp == 2 && lane < ctas && cta->abort)
        st_cluster_int(mapa_shared(smem_u32(const_cast<int*>(&cta->abort)), lane), 1);
      __syncwarp();
      cluster_sync();
    }
  } else {
    // ---------------- sums and outputs ----------------
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    float acc[Sh::PARTS][Sh::HALF];
#pragma unroll
    for (int p = 0; p < Sh::PARTS; ++p)
#pragma unroll
      for (int i = 0; i < Sh::HALF; ++i) acc[p][i] = 0.f;
    if (!GATED && g.o.add[problem]) {
      // this CTA's part of the addend comes into L2 while the products run: a thread takes half of a row's 128 columns
      const int size = g.o.out_f32 ? 4 : 2, t = threadIdx.x - 128, per = BN >> g.k_log;
      const int64_t r = static_cast<int64_t>(qb) * BN + rank * per + (t >> 1), c = static_cast<int64_t>(pb) * 128 + (t & 1) * 64;
      if ((t >> 1) < per && r < g.rows && c < g.cols) {
        const uint8_t* at = static_cast<const uint8_t*>(g.o.add[problem]) + (r * g.o.ld_add[problem] + c) * size;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        if (size == 4 && c + 32 < g.cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 128));
      }
    }
    int a = 0;
    uint32_t aph = 0;
    bool ok = true;
#pragma unroll 1
    for (int kc = k0; kc < k1; kc += g.restart) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar->acc_full[a], aph, g.ctl, cta, kSiteEpilogueAccFull));
      if (!ok) break;
      tc_fence_after();
      const uint32_t src = tmem + lanes + a * Sh::PARTS * BN + half * Sh::HALF;
#pragma unroll
      for (int p = 0; p < Sh::PARTS; ++p) {
#pragma unroll
        for (int j = 0; j < Sh::HALF; j += 8) {
          uint32_t v[8];
          tmem_ld_few(src + p * BN + j, v);
          tmem_wait_ld();
          regs_after_wait(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[p][j + i] += __uint_as_float(v[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->acc_empty[a]);
      if (++a == 2) { a = 0; aph ^= 1u; }
    }
    // The ring has served its last K block, in every CTA of the cluster after
    // this: its memory takes the sums.
    if (ctas > 1)
      cluster_sync();
    else
      asm volatile("bar.sync 1, %0;" ::"n"(kFewAddThreads) : "memory");
    const int per = BN >> g.k_log;    // of q's rows per CTA
    const uint32_t at = smem_u32(ring) + (static_cast<int>(rank) * per * kFewRow + row) * 4;
    const int there = g.rows - qb * BN;   // of q's rows
    // 32 lanes' sums of one of q's rows lie side by side
#pragma unroll
    for (int p = 0; p < Sh::PARTS; ++p) {
#pragma unroll
      for (int i = 0; i < Sh::HALF; ++i) {
        const int col = half * Sh::HALF + i;
        if (col >= there) break;
        const uint32_t here = at + (p * BN + (col & (per - 1))) * (kFewRow * 4);
        if (ctas > 1)
          st_cluster_f1(mapa_shared(here, static_cast<uint32_t>(col / per)), acc[p][i]);
        else
          st_shared_f1(here, acc[p][i]);
      }
    }
    if (ctas > 1)
      cluster_sync();
    else
      asm volatile("bar.sync 1, %0;" ::"n"(kFewAddThreads) : "memory");
    if (ok && !cta->abort) {
      const float* buf = reinterpret_cast<const float*>(ring);
      const int t = threadIdx.x - 128;
      const int64_t col0 = static_cast<int64_t>(pb) * 128, row0 = static_cast<int64_t>(qb) * BN + rank * per;
      if (g.o.bf16) {
        if (!GATED && g.o.out_f32)
          finish_few<BN, GATED, __nv_bfloat16, float>(g, problem, buf, t, ctas, per, row0, col0);
        else
          finish_few<BN, GATED, __nv_bfloat16, __nv_bfloat16>(g, problem, buf, t, ctas, per, row0, col0);
      } else {
        if (!GATED && g.o.out_f32)
          finish_few<BN, GATED, __half, float>(g, problem, buf, t, ctas, per, row0, col0);
        else
          finish_few<BN, GATED, __half, __half>(g, problem, buf, t, ctas, per, row0, col0);
      }
    }
  }

  __syncthreads();
  if (cta->abort && prod.which >= 0 && lane == 0) prod.drain(bar->full, Sh::STAGES, g.ctl);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

template <int BN, bool GATED, bool P_MN, bool Q_MN>
cudaError_t launch_as(FfnProduct& p, const void** kernel) {
  using Sh = FewShape<BN, GATED>;
  static_assert(!Q_MN || BN >= 64, "a row of an MN-major box is 64 of the operand's rows");
  auto k = ffn_few_kernel<BN, GATED, P_MN, Q_MN>;
  *kernel = reinterpret_cast<const void*>(k);
  const bool sum = p.op == kFfnInputGrad && p.count == 2, both = p.op == kFfnWeightGrad && p.count == 2;
  FewMaps maps = {};
  cudaError_t e;
  if (p.summed > 0) {
    for (int i = 0; i < (sum || both ? 2 : 1); ++i) {
      e = Q_MN && BN == 64 ? cudaSuccess : ffn_map(&maps.q[i], p, p.a[i], p.lda[i], p.rows, Q_MN, BN);
      if (e == cudaSuccess && Q_MN) e = ffn_map64(&maps.q64[i], p, p.a[i], p.lda[i], p.rows, true);
      if (e != cudaSuccess) return e;
    }
    for (int i = 0; i < (sum || GATED ? 2 : 1); ++i) {
      e = ffn_map(&maps.p[i], p, p.b[i], p.ldb[i], p.cols, P_MN, 128);
      if (e == cudaSuccess && P_MN && p.cols % 64 != 0) e = ffn_map64(&maps.p64[i], p, p.b[i], p.ldb[i], p.cols, true);
      if (e != cudaSuccess) return e;
    }
  }
  FewParams g = {};
  g.o = p.out;
  g.rows = static_cast<int32_t>(p.rows);
  g.cols = static_cast<int32_t>(p.cols);
  g.kt = static_cast<int32_t>((p.summed + kFfnBK - 1) / kFfnBK);
  g.sources = sum ? 2 : 1;
  g.problems = both ? 2 : 1;
  g.restart = ffn_restart(p.out.out_f32 != 0, p.out.bf16 != 0);
  g.k_log = p.plan.k_splits == 8 ? 3 : (p.plan.k_splits == 4 ? 2 : (p.plan.k_splits == 2 ? 1 : 0));
  g.row_blocks = (g.rows + BN - 1) / BN;
  g.per_problem = g.row_blocks * ((g.cols + 127) / 128);
  g.idesc = umma_idesc_f16(p.out.bf16 != 0, 128, BN) | (P_MN ? kIdescAMn : 0u) | (Q_MN ? kIdescBMn : 0u);
  g.ctl = p.ctl;
  if ((e = ensure_smem_attr(*kernel, Sh::SMEM)) != cudaSuccess) return e;
  RingConfig c(p.plan.grid, kFewThreads, p.plan.k_splits, Sh::SMEM, p.stream);
  return cudaLaunchKernelEx(&c.cfg, k, maps, g);
}

template <int BN, bool GATED>
void shape_of(gp_plan* p) {
  using Sh = FewShape<BN, GATED>;
  p->stages = Sh::STAGES;
  p->stage_bytes = Sh::STAGE;
  p->ring_bytes = Sh::STAGES * Sh::STAGE;
  p->smem_bytes = Sh::SMEM;
  p->tmem_cols = Sh::TMEM_COLS;
  p->threads = kFewThreads;
}

}  // namespace

int ffn_few_most_ctas(int rows) { return rows == 16 ? 4 : 8; }

void ffn_few_shape(gp_plan* p, int rows, bool gated) {
  switch (rows) {
    case 16: return gated ? shape_of<16, true>(p) : shape_of<16, false>(p);
    case 32: return gated ? shape_of<32, true>(p) : shape_of<32, false>(p);
    case 64: return gated ? shape_of<64, true>(p) : shape_of<64, false>(p);
    default: return shape_of<128, false>(p);
  }
}

namespace {

template <bool P_MN>
cudaError_t launch_rows(FfnProduct& p, const void** kernel) {
  switch (p.plan.bn) {
    case 16: return launch_as<16, false, P_MN, false>(p, kernel);
    case 32: return launch_as<32, false, P_MN, false>(p, kernel);
    case 64: return launch_as<64, false, P_MN, false>(p, kernel);
    default: return launch_as<128, false, P_MN, false>(p, kernel);
  }
}

}  // namespace

cudaError_t launch_ffn_few(FfnProduct& p, const void** kernel) {
  switch (p.op) {
    case kFfnLinear: return launch_rows<false>(p, kernel);
    case kFfnInputGrad: return launch_rows<true>(p, kernel);
    case kFfnGated:
      return p.plan.bn == 16   ? launch_as<16, true, false, false>(p, kernel)
             : p.plan.bn == 32 ? launch_as<32, true, false, false>(p, kernel)
                               : launch_as<64, true, false, false>(p, kernel);
    default: return p.plan.bn == 64 ? launch_as<64, false, true, true>(p, kernel) : launch_as<128, false, true, true>(p, kernel);
  }
}

}  // namespace gp
