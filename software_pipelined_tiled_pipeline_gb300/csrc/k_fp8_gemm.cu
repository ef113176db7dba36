// k_fp8_gemm.cu -- C = A x B^T of 8-bit matrices with an FP32 scale for each
// 128 values along K (and for each row, or each 128 rows), on the tensor cores.
//
//   C[m][n] = sum over K blocks b of  sA[m][b] * sB[n][b] * (sum over the 128 k of b of a[m][k] * b[n][k])
//
// The inner sums are tcgen05.mma (kind::f8f6f4, FP32 accumulators in TMEM),
// restarted for each K block; the outer sum is FP32 in registers, one FMA per
// output and K block: acc = fma(d, sP * sQ, acc).  Persistent and
// warp-specialised, 12 warps per CTA:
//   warp 0      TMA producer: one ring slot = one K block = 128 bytes of each row
//   warp 1      allocates TMEM, issues the MMAs of a K block into the next TMEM
//               buffer, releases the slot and signals the buffer
//   warp 2      brings the K block's scales into a small ring (cp.async)
//   warps 4-11  add each TMEM buffer, scaled, to the sums in their registers;
//               at a tile's end they write C
// Warp w may read TMEM lanes 32 (w mod 4) .. +31; the two warps of a quarter
// take half the columns each.  "P" is the operand on the MMA's M side (128
// rows per CTA), "Q" the one on its N side (BN rows); either may be A.
#include <cstring>
#include "fp8_internal.h"
#include "gp_device.cuh"

namespace gp {
namespace {

constexpr int kBK = 128;                  // K block: bytes of a row per ring slot, and values per scale
constexpr int kMmaK = 32;                 // K of one kind::f8f6f4 instruction
constexpr int kThreads = 384;
constexpr int kAddWarps = 8;
constexpr int kScaleSlots = 8;
constexpr int kStageWarpBytes = 32 * 128;   // output staging of one warp: 32 rows of 32 FP32
constexpr int kMaxRing = 12;
constexpr int64_t kMaxTiles = int64_t(1) << 30;   // tile numbers plus a grid stay below 2^31

struct Fp8Barriers {
  uint64_t full[kMaxRing];
  uint64_t empty[kMaxRing];
  uint64_t acc_full[8];
  uint64_t acc_empty[8];
  uint64_t sc_full[kScaleSlots];
  uint64_t sc_empty[kScaleSlots];
  uint64_t drain;
  uint32_t tmem_base;
  int32_t consumed_hi;       // K blocks that the MMA thread has taken (low 31 bits)
  CtaCtl ctl;
  int32_t last;              // this CTA completed the last segment of a split tile
};
constexpr int kFp8BarrierBytes = 576;
static_assert(sizeof(Fp8Barriers) <= kFp8BarrierBytes, "barrier region too small");

template <int BN>
struct Fp8Shape {
  static constexpr int P_ROWS = 128;
  static constexpr int Q_ROWS = BN;
  static constexpr int TILE_P = 128;
  static constexpr int P_BYTES = P_ROWS * kBK;
  static constexpr int STAGE = (P_ROWS + Q_ROWS) * kBK;
  static constexpr int BUFS = BN == 256 ? 2 : (BN == 128 ? 4 : 8);   // TMEM accumulators
  static constexpr uint32_t TMEM_COLS = BUFS * BN;
  static constexpr int HALF = BN / 2;                  // columns per adding warp
  static constexpr int SCALES = P_ROWS + BN;           // floats per scale slot
  static constexpr int FIXED = kAddWarps * kStageWarpBytes + kScaleSlots * SCALES * 4 + kFp8BarrierBytes + 1024;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kMaxRing ? FIT : kMaxRing;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
};

// One operand's scales: element (row, block) at base[(row / group) * stride_row + block * stride_col].
struct ScaleView {
  const float* base;
  int64_t stride_row, stride_col;
  int32_t rows;              // rows of the operand
  int32_t shift;             // 0 or 7: log2 of the group
};

struct Fp8Params {
  ScaleView p, q;
  void* c;
  const void* addend;
  int64_t ldc, ld_add;
  int32_t K;
  int32_t out_type;
  int32_t swapped;           // P is B: C's rows run along Q
  int32_t vec;               // groups of 4 outputs are aligned to their size
  uint32_t idesc;
  int32_t raster_gp;         // P blocks per raster group
  KernelCtl ctl;
};

// Instruction descriptor of kind::f8f6f4 with FP32 accumulation, both operands
// K-major: D format F32 (bits 4-5 = 1), A and B format (bits 7-9, 10-12: 0 =
// E4M3, 1 = E5M2), N >> 3 (bits 17-22), M >> 4 (bits 24-28).
uint32_t idesc_f8(int p_format, int q_format, uint32_t m, uint32_t n) {
  return (1u << 4) | (static_cast<uint32_t>(p_format) << 7) | (static_cast<uint32_t>(q_format) << 10) |
         ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[8]) { tmem_ld_32x32b_x8(t, r); }
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(t, r); }
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(t, r); }

// 4 bytes from global to shared memory without a register; zeros where !valid (nothing is read then).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
// Arrive on bar when this thread's copies so far have landed (counts against the barrier's count).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Wait of a whole warp; false in every lane if it gave up in one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const KernelCtl& ctl, CtaCtl* cta,
                                          uint32_t site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, cta, site));
}

// Output tile -> its P and Q blocks: groups of `gp` P blocks, each swept over all Q blocks.
__device__ __forceinline__ void tile_blocks(int tile, int p_blocks, int q_blocks, int gp, int& pb, int& qb) {
  const int per = gp * q_blocks;
  const int group = tile / per;
  const int first = group * gp;
  const int n = min(gp, p_blocks - first);
  const int in = tile - group * per;
  pb = first + in % n;
  qb = in / n;
}

// Four neighbouring outputs of a row: FP32 sums (+ addend) rounded to the output type.
template <typename T>
__device__ __forceinline__ void store4(const Fp8Params& g, float4 v, int64_t row, int64_t col, int64_t cols) {
  T* c = static_cast<T*>(g.c) + row * g.ldc + col;
  const T* add = g.addend ? static_cast<const T*>(g.addend) + row * g.ld_add + col : nullptr;
  float x[4] = {v.x, v.y, v.z, v.w};
  struct alignas(4 * sizeof(T)) Four { T e[4]; };
  auto widen = [](T t) {
    if constexpr (sizeof(T) == 4) return t; else return static_cast<float>(t);
  };
  auto narrow = [](float f) {
    if constexpr (sizeof(T) == 4) return f; else return static_cast<T>(f);   // nearest even
  };
  if (g.vec && col + 4 <= cols) {
    if (add) {
      const Four a = *reinterpret_cast<const Four*>(add);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += widen(a.e[i]);
    }
    Four o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.e[i] = narrow(x[i]);
    *reinterpret_cast<Four*>(c) = o;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col + i >= cols) break;
    c[i] = narrow(add ? x[i] + widen(add[i]) : x[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store1(const Fp8Params& g, float v, int64_t row, int64_t col) {
  if (g.addend) v += static_cast<float>(static_cast<const T*>(g.addend)[row * g.ld_add + col]);
  static_cast<T*>(g.c)[row * g.ldc + col] = static_cast<T>(v);
}

// Write a warp's 32 rows x HALF columns of sums (thread: one row) to C.
template <int HALF, typename T>
__device__ __forceinline__ void write_out(const Fp8Params& g, const float (&acc)[HALF], uint8_t* stage, int lane,
                                          int64_t p0, int64_t q0) {
  if (g.swapped) {
    // the lanes' rows are C's columns: each of C's rows gets 32 neighbouring outputs
    const int64_t col = p0 + lane;
    if (col < g.p.rows) {
#pragma unroll
      for (int i = 0; i < HALF; ++i)
        if (q0 + i < g.q.rows) store1<T>(g, acc[i], q0 + i, col);
    }
    return;
  }
  // Through shared memory, so that a row's outputs leave side by side.  16-byte
  // chunk c of row r lies at c ^ (r mod 8).
  constexpr int CW = HALF < 32 ? HALF : 32;      // columns staged at a time
  constexpr int PER = CW / 4;                    // lanes per row when they leave
  const uint32_t base = smem_u32(stage);
#pragma unroll
  for (int j = 0; j < HALF / CW; ++j) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(base + sw128_offset(lane, i)),
                   "f"(acc[j * CW + 4 * i]), "f"(acc[j * CW + 4 * i + 1]), "f"(acc[j * CW + 4 * i + 2]),
                   "f"(acc[j * CW + 4 * i + 3])
                   : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = i * (32 / PER) + lane / PER, ch = lane % PER;
      float4 v;
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(base + sw128_offset(r, ch))
                   : "memory");
      const int64_t col = q0 + j * CW + 4 * ch;
      if (p0 + r < g.p.rows && col < g.q.rows) store4<T>(g, v, p0 + r, col, g.q.rows);
    }
  }
}

// QROWS: Q has a scale for each row (a column of the tile); else one for each 128 rows.
template <int BN, bool QROWS>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_ring_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ Fp8Params g) {
  using Sh = Fp8Shape<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + Sh::STAGES * Sh::STAGE;
  float* scales = reinterpret_cast<float*>(staging + kAddWarps * kStageWarpBytes);
  Fp8Barriers* bar = reinterpret_cast<Fp8Barriers*>(scales + kScaleSlots * Sh::SCALES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int p_blocks = (g.p.rows + Sh::TILE_P - 1) / Sh::TILE_P;
  const int q_blocks = (g.q.rows + BN - 1) / BN;
  const int tiles = p_blocks * q_blocks;
  const int kt = (g.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Sh::STAGES; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int a = 0; a < Sh::BUFS; ++a) {
      mbar_init(&bar->acc_full[a], 1);
      mbar_init(&bar->acc_empty[a], kAddWarps);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&bar->sc_full[s], 32);
      mbar_init(&bar->sc_empty[s], kAddWarps);
    }
    mbar_init(&bar->drain, 1);
    bar->ctl.abort = 0;
    bar->consumed_hi = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, Sh::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem = bar->tmem_base;
  CtaCtl* cta = &bar->ctl;
  int issued = 0;   // producer only

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        int pb, qb;
        tile_blocks(tile, p_blocks, q_blocks, g.raster_gp, pb, qb);
        for (int kb = 0; kb < kt; ++kb) {
          if (!mbar_wait(&bar->empty[s], ph ^ 1u, g.ctl, cta, kSiteProducerEmpty)) { ok = false; break; }
          uint8_t* slot = ring + s * Sh::STAGE;
          if (!(g.ctl.inject_lost_load && tile == tiles - 1 && kb == kt - 1)) {
            mbar_arrive_expect_tx(&bar->full[s], Sh::STAGE);
            tma_load_2d(smem_u32(slot), &tmP, &bar->full[s], kb * kBK, pb * Sh::TILE_P);
            tma_load_2d(smem_u32(slot + Sh::P_BYTES), &tmQ, &bar->full[s], kb * kBK, qb * BN);
            ++issued;
          }
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      int consumed = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        for (int kb = 0; kb < kt; ++kb) {
          if (!mbar_wait(&bar->acc_empty[a], aph ^ 1u, g.ctl, cta, kSiteMmaAccEmpty) ||
              !mbar_wait(&bar->full[s], ph, g.ctl, cta, kSiteConsumerFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t addr = smem_u32(ring + s * Sh::STAGE);
          const uint64_t dp = umma_desc_sw128(addr);
          const uint64_t dq = umma_desc_sw128(addr + Sh::P_BYTES);
          const uint32_t d = tmem + a * BN;
#pragma unroll
          for (int kk = 0; kk < kBK / kMmaK; ++kk)   // 32 bytes along K: the start address field moves by 2
            umma_f8(d, dp + 2 * kk, dq + 2 * kk, g.idesc, kk == 0 ? 0u : 1u);
          umma_commit(&bar->empty[s]);
          umma_commit(&bar->acc_full[a]);
          ++consumed;
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
          if (++a == Sh::BUFS) { a = 0; aph ^= 1u; }
        }
      }
      bar->consumed_hi = consumed;
      umma_commit(&bar->drain);   // fires when every MMA issued above has completed
      CtaCtl never_abort{0};
      mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
    }
  } else if (warp == 2) {
    // ---------------- scales ----------------
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      int pb, qb;
      tile_blocks(tile, p_blocks, q_blocks, g.raster_gp, pb, qb);
      for (int kb = 0; kb < kt; ++kb) {
        if (!warp_wait(&bar->sc_empty[s], ph ^ 1u, g.ctl, cta, kSiteProducerEmpty)) { ok = false; break; }
        const uint32_t dst = smem_u32(scales + s * Sh::SCALES);
        const float* pk = g.p.base + kb * g.p.stride_col;
        const float* qk = g.q.base + kb * g.q.stride_col;
#pragma unroll
        for (int i = 0; i < Sh::P_ROWS / 32; ++i) {
          const int r = i * 32 + lane;
          const int64_t row = static_cast<int64_t>(pb) * Sh::TILE_P + r;
          const bool in = row < g.p.rows;
          cp_async4(dst + r * 4, in ? pk + (row >> g.p.shift) * g.p.stride_row : pk, in);
        }
        if (QROWS) {
#pragma unroll
          for (int i = 0; i < (BN + 31) / 32; ++i) {
            const int r = i * 32 + lane;
            const int64_t row = static_cast<int64_t>(qb) * BN + r;
            const bool in = r < BN && row < g.q.rows;
            if (r < BN) cp_async4(dst + (Sh::P_ROWS + r) * 4, in ? qk + (row >> g.q.shift) * g.q.stride_row : qk, in);
          }
        } else if (lane < (BN + 127) / 128) {
          const int64_t row = static_cast<int64_t>(qb) * BN + lane * 128;
          const bool in = row < g.q.rows;
          cp_async4(dst + (Sh::P_ROWS + lane) * 4, in ? qk + (row >> g.q.shift) * g.q.stride_row : qk, in);
        }
        cp_async_arrive(&bar->sc_full[s]);
        if (++s == kScaleSlots) { s = 0; ph ^= 1u; }
      }
    }
    cp_async_wait_all();
  } else if (warp >= 4) {
    // ---------------- scaled sums and output ----------------
    const int e = warp - 4;
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int half = e >> 2;               // which half of the columns
    const int row = quarter * 32 + lane;   // row of the tile that this thread holds
    uint8_t* my_stage = staging + e * kStageWarpBytes;
    constexpr int CW = Sh::HALF < 32 ? Sh::HALF : 32;
    constexpr int CHUNKS = Sh::HALF / CW;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int a = 0, sc = 0;
    uint32_t aph = 0, sph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      float acc[Sh::HALF];
#pragma unroll
      for (int i = 0; i < Sh::HALF; ++i) acc[i] = 0.f;
      for (int kb = 0; kb < kt; ++kb) {
        ok = warp_wait(&bar->sc_full[sc], sph, g.ctl, cta, kSiteConsumerFull) &&
             warp_wait(&bar->acc_full[a], aph, g.ctl, cta, kSiteEpilogueAccFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + lanes + a * BN + half * Sh::HALF;
        uint32_t v[2][CW];
        tmem_ld(src, v[0]);
        const float* slot = scales + sc * Sh::SCALES;
        const float sp = slot[row];
        const float* sq = slot + Sh::P_ROWS;
        const float both = QROWS ? 0.f : sp * sq[BN == 256 ? half : 0];
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
          tmem_wait_ld();
          regs_after_wait(v[j & 1]);
          if (j + 1 < CHUNKS) {
            tmem_ld(src + (j + 1) * CW, v[(j + 1) & 1]);
          } else {
            // the buffer is in registers: hand it back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar->acc_empty[a]);
          }
          if (QROWS) {
            const float4* q4 = reinterpret_cast<const float4*>(sq + half * Sh::HALF + j * CW);
#pragma unroll
            for (int i = 0; i < CW / 4; ++i) {
              const float4 q = q4[i];
              float* o = acc + j * CW + 4 * i;
              const uint32_t* d = v[j & 1] + 4 * i;
              o[0] = fmaf(__uint_as_float(d[0]), sp * q.x, o[0]);
              o[1] = fmaf(__uint_as_float(d[1]), sp * q.y, o[1]);
              o[2] = fmaf(__uint_as_float(d[2]), sp * q.z, o[2]);
              o[3] = fmaf(__uint_as_float(d[3]), sp * q.w, o[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) acc[j * CW + i] = fmaf(__uint_as_float(v[j & 1][i]), both, acc[j * CW + i]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->sc_empty[sc]);
        if (++a == Sh::BUFS) { a = 0; aph ^= 1u; }
        if (++sc == kScaleSlots) { sc = 0; sph ^= 1u; }
      }
      if (!ok) break;
      int pb, qb;
      tile_blocks(tile, p_blocks, q_blocks, g.raster_gp, pb, qb);
      const int64_t p0 = static_cast<int64_t>(pb) * Sh::TILE_P + quarter * 32;
      const int64_t q0 = static_cast<int64_t>(qb) * BN + half * Sh::HALF;
      if (g.out_type == GP_REAL_BF16)
        write_out<Sh::HALF, __nv_bfloat16>(g, acc, my_stage, lane, p0, q0);
      else if (g.out_type == GP_REAL_F16)
        write_out<Sh::HALF, __half>(g, acc, my_stage, lane, p0, q0);
      else
        write_out<Sh::HALF, float>(g, acc, my_stage, lane, p0, q0);
    }
  }

  __syncthreads();
  if (cta->abort && warp == 0 && lane == 0) {
    // loads still in flight land in shared memory: wait for them before exit
    CtaCtl never_abort{0};
    for (int i = bar->consumed_hi; i < issued; ++i)
      mbar_wait(&bar->full[i % Sh::STAGES], static_cast<uint32_t>((i / Sh::STAGES) & 1), g.ctl, &never_abort,
                kSiteDrain);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

// C = addend or zeros, rows x cols with an ld.
template <typename T>
__global__ void __launch_bounds__(256) fill_kernel(T* c, int64_t ldc, const T* add, int64_t ld_add, int64_t rows,
                                                   int64_t cols) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t n = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / cols, k = i - r * cols;
    c[r * ldc + k] = add ? add[r * ld_add + k] : T(0.f);
  }
}

template <int BN, bool QROWS>
cudaError_t launch_ring(Fp8GemmArgs& a, const void** kernel) {
  using Sh = Fp8Shape<BN>;
  const bool swapped = a.plan.layout != 0;
  const gp_fp8_matrix& P = swapped ? a.B : a.A;
  const gp_fp8_matrix& Q = swapped ? a.A : a.B;
  const int32_t p_rows = swapped ? a.N : a.M, q_rows = swapped ? a.M : a.N;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tmP, tmQ;
  cudaError_t e;
  if ((e = make_tmap_2d(&tmP, P.data, u8, a.K, p_rows, P.ld, kBK, Sh::P_ROWS, CU_TENSOR_MAP_SWIZZLE_128B)) !=
      cudaSuccess)
    return e;
  if ((e = make_tmap_2d(&tmQ, Q.data, u8, a.K, q_rows, Q.ld, kBK, Sh::Q_ROWS, CU_TENSOR_MAP_SWIZZLE_128B)) !=
      cudaSuccess)
    return e;
  Fp8Params g = {};
  g.p = ScaleView{P.scales, P.stride_row, P.stride_col, p_rows, P.group == kFp8Group ? 7 : 0};
  g.q = ScaleView{Q.scales, Q.stride_row, Q.stride_col, q_rows, Q.group == kFp8Group ? 7 : 0};
  g.c = a.C;
  g.addend = a.addend;
  g.ldc = a.ldc;
  g.ld_add = a.ld_add;
  g.K = a.K;
  g.out_type = a.out_type;
  g.swapped = swapped;
  const uint64_t four = 4 * real_bytes(a.out_type);
  auto aligned = [&](const void* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % four == 0 && static_cast<uint64_t>(ld) * real_bytes(a.out_type) % four == 0;
  };
  g.vec = aligned(a.C, a.ldc) && (!a.addend || aligned(a.addend, a.ld_add));
  g.idesc = idesc_f8(P.format, Q.format, Sh::TILE_P, BN);
  g.raster_gp = a.plan.raster_gm;
  g.ctl = a.ctl;
  auto k = fp8_ring_kernel<BN, QROWS>;
  *kernel = reinterpret_cast<const void*>(k);
  if ((e = ensure_smem_attr(*kernel, Sh::SMEM)) != cudaSuccess) return e;
  return launch_dependent(k, dim3(a.plan.grid), dim3(kThreads), Sh::SMEM, a.stream, tmP, tmQ, g);
}

template <int BN>
void shape_of(gp_plan* p) {
  using Sh = Fp8Shape<BN>;
  p->bm = Sh::TILE_P;
  p->bn = BN;
  p->bk = kBK;
  p->stages = Sh::STAGES;
  p->stage_bytes = Sh::STAGE;
  p->ring_bytes = Sh::STAGES * Sh::STAGE;
  p->smem_bytes = Sh::SMEM;
  p->tmem_cols = Sh::TMEM_COLS;
}

}  // namespace

int fp8_plan_impl(int64_t M, int64_t N, int64_t K, int a_group, int b_group, int sms, const gp_fp8_options* opts,
                  gp_plan* p) {
  std::memset(p, 0, sizeof(*p));
  const int want = opts ? opts->bn : 0;
  if (want != 0 && want != 16 && want != 32 && want != 64 && want != 128) return GP_ERR_UNSUPPORTED;
  // Q, the operand on the MMA's N side, is the narrower one where that is at
  // most one tile wide; else the one with block scales (one product of scales
  // per row instead of one per output), B if both or neither.
  const int64_t narrow = M < N ? M : N;
  bool swapped;
  if (narrow <= 128)
    swapped = M < N;
  else
    swapped = a_group == kFp8Group && b_group == 1;
  const int64_t p_rows = swapped ? N : M, q_rows = swapped ? M : N;
  int bn = want;
  if (bn == 0) bn = narrow <= 16 ? 16 : (narrow <= 32 ? 32 : (narrow <= 64 ? 64 : 128));
  p->dtype = GP_PLAN_FP8;
  p->layout = swapped;
  p->variant = GP_PIPELINED;
  p->threads = kThreads;
  p->persistent = 1;
  p->kernel = "fp8_ring";
  switch (bn) {
    case 16: shape_of<16>(p); break;
    case 32: shape_of<32>(p); break;
    case 64: shape_of<64>(p); break;
    default: shape_of<128>(p); break;
  }
  p->tiles = (p_rows + p->bm - 1) / p->bm * ((q_rows + p->bn - 1) / p->bn);
  p->k_tiles = (K + kBK - 1) / kBK;
  if (p->tiles > kMaxTiles) return GP_ERR_SIZE;
  p->grid = sms > 0 ? static_cast<int32_t>(p->tiles < sms ? p->tiles : sms) : 0;
  p->dp_tiles = static_cast<int32_t>(p->tiles);
  p->k_splits = 1;
  p->raster_gm = 8;
  p->compute_load_ratio = 2.0 * p->bm * p->bn / (p->bm + p->bn);
  return GP_OK;
}

cudaError_t launch_fp8_gemm(Fp8GemmArgs& a, const void** kernel) {
  const gp_fp8_matrix& Q = a.plan.layout ? a.A : a.B;
  switch (a.plan.bn) {
    case 16: return launch_ring<16, true>(a, kernel);
    case 32: return launch_ring<32, true>(a, kernel);
    case 64: return launch_ring<64, true>(a, kernel);
    default: return Q.group == 1 ? launch_ring<128, true>(a, kernel) : launch_ring<128, false>(a, kernel);
  }
}

cudaError_t launch_fp8_fill(void* C, int64_t ldc, const void* addend, int64_t ld_add, int64_t M, int64_t N,
                            int out_type, cudaStream_t stream) {
  const int64_t blocks = (M * N + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), block(256);
  switch (out_type) {
    case GP_REAL_F16:
      return launch_dependent(fill_kernel<__half>, grid, block, 0, stream, static_cast<__half*>(C), ldc,
                              static_cast<const __half*>(addend), ld_add, M, N);
    case GP_REAL_BF16:
      return launch_dependent(fill_kernel<__nv_bfloat16>, grid, block, 0, stream, static_cast<__nv_bfloat16*>(C), ldc,
                              static_cast<const __nv_bfloat16*>(addend), ld_add, M, N);
    default:
      return launch_dependent(fill_kernel<float>, grid, block, 0, stream, static_cast<float*>(C), ldc,
                              static_cast<const float*>(addend), ld_add, M, N);
  }
}

}  // namespace gp
