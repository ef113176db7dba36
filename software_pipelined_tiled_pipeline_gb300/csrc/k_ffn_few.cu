// k_ffn_few.cu -- the forward products for few tokens: the weight fills the
// tensor cores' M side (128 rows per CTA), the tokens their N side (16, 32 or
// 64), and a cluster of 1 to 8 CTAs shares a tile's K blocks.
//
//   s[n][m] = sum over k of w[n][k] * x[m][k]
//   linear: out = act(s + bias) + addend;  gated: out = act(g) * u, with a second weight and sums u
//
// The sums of a cluster meet in distributed shared memory: each CTA is handed
// its share of the token columns by all, adds them in K order and writes them.
// What bounds it: the weights' bytes, and for one token the launch, the first
// loads and the exchange.
#include "ffn_ring.cuh"

namespace gp {
namespace {

constexpr int kFewThreads = 384;
constexpr int kFewAddThreads = 256;      // eight warps: 32 rows of the weight x half of the tokens each
constexpr int kFewMaxRing = 12;
constexpr int kFewXRow = 129;            // floats per column of the exchange: keeps either walk off each other's banks

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

template <int BN, bool GATED>
struct FewShape {
  static constexpr int PARTS = GATED ? 2 : 1;
  static constexpr int W_BYTES = 128 * kFfnBK * 2;
  static constexpr int STAGE = PARTS * W_BYTES + BN * kFfnBK * 2;
  static constexpr int FIXED = kFewBarrierBytes + kSmemAlignSlack;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kFewMaxRing ? FIT : kFewMaxRing;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static constexpr uint32_t TMEM_COLS = 2 * PARTS * BN;
  static constexpr int HALF = BN / 2;
  static_assert(PARTS * BN * kFewXRow * 4 <= STAGES * STAGE, "the exchange takes the ring's memory");
  static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS >= 32 && TMEM_COLS <= 512, "TMEM columns");
};

struct FewParams {
  FfnOut o;
  int32_t tokens, n;         // rows and columns of the output
  int32_t kt;
  int32_t restart;
  int32_t k_log;             // log2 of the CTAs that share a tile's K blocks
  int32_t token_blocks;
  uint32_t idesc;
  KernelCtl ctl;
};

struct FewMaps {
  CUtensorMap x, w[2];
};

__device__ __forceinline__ void tmem_ld_few(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void st_cluster_float(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_int(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// The tokens col0 .. of a tile from the exchanged sums of `ctas` CTAs.
template <int BN, bool GATED, typename T, typename O>
__device__ __forceinline__ void finish_few(const FewParams& g, const float* buf, int t, int ctas, int per, int64_t n0,
                                           int64_t m0) {
  const FfnOut& o = g.o;
  const O* const add = static_cast<const O*>(o.add[0]);
  O* const out = static_cast<O*>(o.out[0]);
  T* const keep0 = static_cast<T*>(o.keep[0]);
  T* const keep1 = static_cast<T*>(o.keep[1]);
  const int row = t & 127;
  const int64_t n = n0 + row;
  if (n >= g.n) return;
  float bias = 0.f;
  if (!GATED && o.bias) bias = o.bias_f32 ? static_cast<const float*>(o.bias)[n] : to_f32(static_cast<const T*>(o.bias)[n]);
#pragma unroll 2
  for (int c = t >> 7; c < per; c += kFewAddThreads / 128) {
    const int64_t m = m0 + c;
    if (m >= g.tokens) return;
    float v[1] = {0.f}, u = 0.f;
    O was;
    if (!GATED && add) was = add[m * o.ld_add[0] + n];
    for (int s = 0; s < ctas; ++s) {   // in K order
      v[0] += buf[(s * per + c) * kFewXRow + row];
      if (GATED) u += buf[(BN + s * per + c) * kFewXRow + row];
    }
    v[0] += bias;
    if (keep0) {
      from_f32(v[0], keep0[m * o.ld_keep[0] + n]);
      if (GATED) from_f32(u, keep1[m * o.ld_keep[1] + n]);
    }
    activate_all(v, o.act);
    if (GATED) v[0] *= u;
    if (!GATED && add) v[0] += to_f32(was);
    from_f32(v[0], out[m * o.ld_out[0] + n]);
  }
}

template <int BN, bool GATED>
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
  // token blocks of one weight block side by side: its rows are read from L2 after the first
  const int wb = tile / g.token_blocks, mb = tile - wb * g.token_blocks;
  const int k0 = static_cast<int>((static_cast<int64_t>(g.kt) * rank) >> g.k_log);
  const int k1 = static_cast<int>((static_cast<int64_t>(g.kt) * (rank + 1)) >> g.k_log);

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
  if (warp == 0 && lane == 0) {
    for (int kb = k0; kb < k1 && kb < k0 + Sh::STAGES; ++kb) {
      tma_prefetch_l2_2d(&maps.w[0], kb * kFfnBK, wb * 128);
      if (GATED) tma_prefetch_l2_2d(&maps.w[1], kb * kFfnBK, wb * 128);
      tma_prefetch_l2_2d(&maps.x, kb * kFfnBK, mb * BN);
    }
  }
  pdl_wait();
  const uint32_t tmem = bar->tmem_base;
  CtaCtl* cta = &bar->ctl;
  int issued = 0, lost = -1;

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // ---------------- producer ----------------
      const bool lose = g.ctl.inject_lost_load && tile == static_cast<int>(gridDim.x >> g.k_log) - 1;
      int s = 0;
      uint32_t ph = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&bar->empty[s], ph ^ 1u, g.ctl, cta, kSiteProducerEmpty) || cta->abort) break;
        const uint32_t at = smem_u32(ring + s * Sh::STAGE);
        if (lose && kb == g.kt - 1) {   // test hook: this load never comes
          lost = issued;
        } else {
          mbar_arrive_expect_tx(&bar->full[s], Sh::STAGE);
          tma_load_2d(at, &maps.w[0], &bar->full[s], kb * kFfnBK, wb * 128);
          if (GATED) tma_load_2d(at + Sh::W_BYTES, &maps.w[1], &bar->full[s], kb * kFfnBK, wb * 128);
          tma_load_2d(at + Sh::PARTS * Sh::W_BYTES, &maps.x, &bar->full[s], kb * kFfnBK, mb * BN);
        }
        ++issued;
        if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      const bool leader = ring_elect_one();
      const uint64_t desc0 = umma_desc_sw128(smem_u32(ring));
      for (int kc = k0; ok && kc < k1; kc += g.restart) {
        const int end = min(kc + g.restart, k1);
        if (!__all_sync(0xffffffffu, mbar_wait(&bar->acc_empty[a], aph ^ 1u, g.ctl, cta, kSiteMmaAccEmpty))) break;
        tc_fence_after();
        const uint32_t d = tmem + a * Sh::PARTS * BN;
        for (int kb = kc; kb < end; ++kb) {
          const bool there = mbar_wait(&bar->full[s], ph, g.ctl, cta, kSiteConsumerFull);
          tc_fence_after();
          const uint64_t dw = desc0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
          const uint64_t dx = dw + Sh::PARTS * Sh::W_BYTES / 16;
          if (leader && there) {
#pragma unroll
            for (int kk = 0; kk < kFfnBK / 16; ++kk) {
              const uint32_t more = kb > kc || kk > 0;
              umma_f16(d, dw + 2 * kk, dx + 2 * kk, g.idesc, more);
              if (GATED) umma_f16(d + BN, dw + Sh::W_BYTES / 16 + 2 * kk, dx + 2 * kk, g.idesc, more);
            }
            umma_commit(&bar->empty[s]);
          }
          if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (leader) umma_commit(&bar->acc_full[a]);
        if (++a == 2) { a = 0; aph ^= 1u; }
      }
      if (leader) {
        umma_commit(&bar->drain);
        CtaCtl never_abort{0};
        mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
      }
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
    const int per = BN >> g.k_log;    // token columns per CTA
    const uint32_t at = smem_u32(ring) + (rank * per * kFewXRow + row) * 4;
#pragma unroll
    for (int p = 0; p < Sh::PARTS; ++p) {
#pragma unroll
      for (int i = 0; i < Sh::HALF; ++i) {
        const int col = half * Sh::HALF + i;
        const uint32_t here = at + (p * BN + (col & (per - 1))) * (kFewXRow * 4);
        if (ctas > 1)
          st_cluster_float(mapa_shared(here, static_cast<uint32_t>(col / per)), acc[p][i]);
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(here), "f"(acc[p][i]) : "memory");
      }
    }
    if (ctas > 1)
      cluster_sync();
    else
      asm volatile("bar.sync 1, %0;" ::"n"(kFewAddThreads) : "memory");
    if (ok && !cta->abort) {
      const float* buf = reinterpret_cast<const float*>(ring);
      const int t = threadIdx.x - 128;
      const int64_t n0 = static_cast<int64_t>(wb) * 128, m0 = static_cast<int64_t>(mb) * BN + rank * per;
      if (g.o.bf16) {
        if (!GATED && g.o.out_f32)
          finish_few<BN, GATED, __nv_bfloat16, float>(g, buf, t, ctas, per, n0, m0);
        else
          finish_few<BN, GATED, __nv_bfloat16, __nv_bfloat16>(g, buf, t, ctas, per, n0, m0);
      } else {
        if (!GATED && g.o.out_f32)
          finish_few<BN, GATED, __half, float>(g, buf, t, ctas, per, n0, m0);
        else
          finish_few<BN, GATED, __half, __half>(g, buf, t, ctas, per, n0, m0);
      }
    }
  }

  __syncthreads();
  if (cta->abort && warp == 0 && lane == 0) {
    // loads still in flight land in shared memory: wait for them before exit
    CtaCtl never_abort{0};
    for (int i = issued > Sh::STAGES ? issued - Sh::STAGES : 0; i < issued; ++i) {
      if (i == lost) continue;
      mbar_wait(&bar->full[i % Sh::STAGES], static_cast<uint32_t>((i / Sh::STAGES) & 1), g.ctl, &never_abort, kSiteDrain);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

template <int BN, bool GATED>
cudaError_t launch_as(FfnProduct& p, const void** kernel) {
  using Sh = FewShape<BN, GATED>;
  auto k = ffn_few_kernel<BN, GATED>;
  *kernel = reinterpret_cast<const void*>(k);
  FewMaps maps = {};
  cudaError_t e;
  if (p.summed > 0) {
    if ((e = ffn_map(&maps.x, p, p.a[0], p.lda[0], p.rows, false, BN)) != cudaSuccess) return e;
    if ((e = ffn_map(&maps.w[0], p, p.b[0], p.ldb[0], p.cols, false, 128)) != cudaSuccess) return e;
    if (GATED && (e = ffn_map(&maps.w[1], p, p.b[1], p.ldb[1], p.cols, false, 128)) != cudaSuccess) return e;
  }
  FewParams g = {};
  g.o = p.out;
  g.tokens = static_cast<int32_t>(p.rows);
  g.n = static_cast<int32_t>(p.cols);
  g.kt = static_cast<int32_t>((p.summed + kFfnBK - 1) / kFfnBK);
  g.restart = p.out.out_f32 ? kFfnRestart : (g.kt > 0 ? g.kt : 1);
  g.k_log = p.plan.k_splits == 8 ? 3 : (p.plan.k_splits == 4 ? 2 : (p.plan.k_splits == 2 ? 1 : 0));
  g.token_blocks = (g.tokens + BN - 1) / BN;
  g.idesc = umma_idesc_f16(p.out.bf16 != 0, 128, BN);
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

void ffn_few_shape(gp_plan* p, int bn, bool gated) {
  if (gated)
    bn == 16 ? shape_of<16, true>(p) : bn == 32 ? shape_of<32, true>(p) : shape_of<64, true>(p);
  else
    bn == 16 ? shape_of<16, false>(p) : bn == 32 ? shape_of<32, false>(p) : shape_of<64, false>(p);
}

cudaError_t launch_ffn_few(FfnProduct& p, const void** kernel) {
  const bool gated = p.op == kFfnGated;
  switch (p.plan.bn) {
    case 16: return gated ? launch_as<16, true>(p, kernel) : launch_as<16, false>(p, kernel);
    case 32: return gated ? launch_as<32, true>(p, kernel) : launch_as<32, false>(p, kernel);
    default: return gated ? launch_as<64, true>(p, kernel) : launch_as<64, false>(p, kernel);
  }
}

}  // namespace gp
