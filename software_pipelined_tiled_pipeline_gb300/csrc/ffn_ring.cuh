// ffn_ring.cuh -- out = a x b^T of 16-bit matrices on the tensor cores, with
// what the feed-forward operators make of the sums on their way out.
//
//   s[r][c] = sum over k of a[r][k] * b[c][k]
//   linear:  z = s + bias;  z may be kept, in 16 bits or in 8;  out = act(z) + addend
//   gated:   b's rows come from two weights, so that a tile holds both sums g and u of
//            the same outputs;  both may be kept;  out = act(g) * u
//   gradients: out = s (+ addend), with a or b stored summed axis first (their
//            columns side by side: "MN major"), so that nothing is transposed in memory
//
// Persistent and warp-specialised:
//   warp 0     TMA producer: one ring slot = 64 of the summed axis
//   warp 1     allocates TMEM and issues tcgen05.mma (kind::f16, FP32 in TMEM)
//   warps 4+   take a tile's sums to registers, 32 rows x 128 columns per warp, hand
//              the TMEM buffer back and write the outputs while the next tile's
//              products run into the other buffer
// PAIR: a cluster of two CTAs shares a 256 x 256 tile (M = 256 instructions).
//
// The tensor cores cut their FP32 sums instead of rounding them, always towards
// zero (measured on normal operands: 1.0e-6 relative after 1024 of K, 9e-6 after
// 8192).  For 16-bit outputs that is far below their rounding (2^-9 on average
// for BF16).  Where FP32 leaves, or the scales of 8-bit codes, the accumulator is
// handed over every kFfnRestart slots (512 of K) and added to sums in registers.
#pragma once
#include <atomic>
#include <cstring>
#include "ffn_math.cuh"
#include "fp8_rows.cuh"
#include "gp_device.cuh"

namespace gp {

constexpr int kRingWarpStage = 32 * 256;   // output staging of one warp: 32 rows of 64 FP32
constexpr int kRingLaunchRegs = 168;       // registers per thread at launch, where warps trade them
constexpr int kRingMax = 8;

struct RingBarriers {
  uint64_t full[kRingMax];
  uint64_t empty[kRingMax];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  CtaCtl ctl;
};
constexpr int kRingBarrierBytes = 256;
static_assert(sizeof(RingBarriers) <= kRingBarrierBytes, "barrier region too small");

template <int BN, bool PAIR>
struct RingShape {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int A_ROWS = 128;                     // per CTA
  static constexpr int B_ROWS = BN / CTAS;
  static_assert(B_ROWS == 128, "a CTA's share of b is two blocks of 64");
  static constexpr int TILE_ROWS = A_ROWS * CTAS;
  static constexpr int A_BYTES = A_ROWS * kFfnBK * 2;
  static constexpr int STAGE = (A_ROWS + B_ROWS) * kFfnBK * 2;
  static constexpr int EPI_WARPS = BN / 32;              // 32 rows x 128 columns each
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr int FIXED = EPI_WARPS * kRingWarpStage + kRingBarrierBytes + kSmemAlignSlack;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kRingMax ? FIT : kRingMax;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  // The warps that write hold 128 sums per thread, and take registers for them
  // from the other four (of a 384-thread launch).
  static constexpr bool SPLIT_REGS = THREADS == 384;
  static constexpr int EPI_REGS = 216, OTHER_REGS = 72;
  static_assert(!SPLIT_REGS || THREADS * kRingLaunchRegs == 32 * (EPI_WARPS * EPI_REGS + 4 * OTHER_REGS), "register split");
};

struct RingParams {
  FfnOut o;
  int32_t rows, cols;        // of the output
  int32_t kt;                // K blocks of one source
  int32_t sources;           // summed one after another
  int32_t problems;          // products in this launch, with operands and outputs of their own
  int32_t restart;           // K blocks per hand-over of the accumulator
  int32_t raster;            // row blocks per raster group
  uint32_t idesc;
  KernelCtl ctl;
};

// Shared-memory descriptor of an MN-major operand tile as TMA copies it with
// 128-byte swizzling: a row of 128 bytes is 64 neighbouring rows of the operand
// at one k, 8 such rows (8 k) 1024 bytes apart (stride byte offset), and the
// next 64 operand rows one box of 64 k further on (leading byte offset 8192).
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((64u * 128u) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptor bits 15 and 16: operand A, B is MN-major.
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

__device__ __forceinline__ bool ring_elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// Arrive on an mbarrier of another CTA of the cluster without ordering memory:
// the TMEM buffer it hands back has been read into registers.
__device__ __forceinline__ void ring_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Output tile -> its row and column blocks: groups of `gp` row blocks, each
// swept over all column blocks, so that CTAs at work at one time share operands in L2.
__device__ __forceinline__ void ring_tile(int tile, int row_blocks, int col_blocks, int gp, int& rb, int& cb) {
  const int per = gp * col_blocks;
  const int group = tile / per;
  const int first = group * gp;
  const int n = min(gp, row_blocks - first);
  const int in = tile - group * per;
  rb = first + in % n;
  cb = in / n;
}

// ---------------------------------------------------------------------------
// sums to outputs: one warp, 32 rows; a thread holds 128 sums of one row
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st_shared_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, float& a, float& b, float& c, float& d) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a), "=f"(b), "=f"(c), "=f"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint4& v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
}

// 16-byte chunk `chunk` of 256-byte row `row` of a warp's staging: rows 0 to 7 at
// one chunk, and chunks at one row, fall on different banks.
__device__ __forceinline__ uint32_t stage_at(uint32_t base, int row, int chunk) {
  return base + static_cast<uint32_t>(row * 256 + ((chunk ^ (row & 15)) << 4));
}

// N neighbouring values of a row on a boundary of their size (16 bytes at most).
template <typename T, int N>
struct alignas(16) RawN {
  T e[N];
};
template <typename T, int N>
__device__ __forceinline__ void load_n(RawN<T, N>& r, const T* p) {
  if constexpr (sizeof(T) * N >= 16) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) * N / 16); ++i)
      reinterpret_cast<uint4*>(r.e)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    *reinterpret_cast<uint2*>(r.e) = *reinterpret_cast<const uint2*>(p);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  RawN<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) from_f32(v[i], r.e[i]);
  if constexpr (sizeof(T) * N >= 16) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) * N / 16); ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(r.e)[i];
  } else {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r.e);
  }
}

// Sixteen codes of a row, as far as its columns go.
__device__ __forceinline__ void store_codes16(uint8_t* row, uint4 v, int64_t col, int64_t cols) {
  if (col + 16 <= cols) {
    *reinterpret_cast<uint4*>(row + col) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (col + i < cols) row[col + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
}

// out = act(s + bias) + addend of 32 rows x 128 columns.  `rows`: rows of the output (0: nothing is written).
template <typename T, typename O>
__device__ __forceinline__ void finish_linear(const RingParams& g, int p, float (&acc)[128], uint8_t* stage, int lane,
                                              int64_t row0, int64_t col0, int64_t rows) {
  const FfnOut& o = g.o;
  const uint32_t base = smem_u32(stage);
  const int64_t cols = g.cols;
  if (col0 >= cols) return;
  if (o.bias) {
    // a lane fetches four columns' bias, all read all of it
    float b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = col0 + 4 * lane + i;
      b[i] = 0.f;
      if (c < cols) b[i] = o.bias_f32 ? static_cast<const float*>(o.bias)[c] : to_f32(static_cast<const T*>(o.bias)[c]);
    }
    __syncwarp();
    st_shared_v4(base + lane * 16, b[0], b[1], b[2], b[3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float x, y, z, w;
      ld_shared_v4(base + i * 16, x, y, z, w);
      acc[4 * i] += x;
      acc[4 * i + 1] += y;
      acc[4 * i + 2] += z;
      acc[4 * i + 3] += w;
    }
  }
  if (o.codes[0].data) {
    // the thread's row has its group of 128 columns to itself
    if (col0 + 128 > cols) {   // (an infinity times a column that is not there is NaN)
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (col0 + i >= cols) acc[i] = 0.f;
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 128; ++i) most = max(most, abs_bits(acc[i]));
    const GroupScale s = group_scale(most, 448.f);
    const FfnCodes& q = o.codes[0];
    if (row0 + lane < rows) q.scales[(row0 + lane) * q.stride_row + (col0 >> 7) * q.stride_col] = s.scale;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float* v = acc + 16 * i + 4 * j;
        w[j] = fp8x4<false>(v[0] * s.inv, v[1] * s.inv, v[2] * s.inv, v[3] * s.inv);
      }
      st_shared_v4(base + sw128_offset(lane, i), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + lane / 8;
      uint4 v;
      ld_shared_v4(base + sw128_offset(r, lane % 8), v);
      if (row0 + r < rows) store_codes16(q.data + (row0 + r) * q.ld, v, col0 + lane % 8 * 16, cols);
    }
  }
  const int lr = lane >> 3, lc = lane & 7;
  const O* const add = static_cast<const O*>(o.add[p]);
  O* const out = static_cast<O*>(o.out[p]);
  T* const keep = static_cast<T*>(o.keep[0]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float* x = acc + j * 64 + 4 * i;
      st_shared_v4(stage_at(base, lane, i), x[0], x[1], x[2], x[3]);
    }
    __syncwarp();
    const int64_t first = col0 + j * 64;
    // eight lanes to a row, eight columns each, where rows are on 16-byte boundaries
    const int64_t col = first + lc * 8;
    const bool mine = o.vec && col + 8 <= cols;
    constexpr int AHEAD = sizeof(O) == 4 ? 2 : 4;   // (more, and registers spill)
#pragma unroll 1
    for (int r0 = lr; r0 < 32; r0 += 4 * AHEAD) {
      RawN<O, 8> was[AHEAD];
      if (add) {
        // addends are asked for before the first of these outputs is written: they may be the same memory
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (mine && row0 + r0 + 4 * u < rows) load_n(was[u], add + (row0 + r0 + 4 * u) * o.ld_add[p] + col);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = r0 + 4 * u;
        float v[8], t[8];
        // (the first of the two chunks alternates, so that eight lanes meet eight banks)
        const int odd = lc >> 2;
        ld_shared_v4(stage_at(base, r, 2 * lc + odd), t[0], t[1], t[2], t[3]);
        ld_shared_v4(stage_at(base, r, 2 * lc + 1 - odd), t[4], t[5], t[6], t[7]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = odd ? t[4 + i] : t[i];
          v[4 + i] = odd ? t[i] : t[4 + i];
        }
        if (!mine || row0 + r >= rows) continue;
        if (keep) store_n(keep + (row0 + r) * o.ld_keep[0] + col, v);
        activate_all(v, o.act);
        if (add) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += to_f32(was[u].e[i]);
        }
        store_n(out + (row0 + r) * o.ld_out[p] + col, v);
      }
    }
    // what is left of a row one by one, a lane to a column
    const int64_t rest = o.vec ? (cols & ~int64_t(7)) : 0, end = cols < first + 64 ? cols : first + 64;
    for (int64_t c = (rest > first ? rest : first) + lane; c < end; c += 32) {
      const int at = static_cast<int>(c - first);
#pragma unroll 4
      for (int r = 0; r < 32; ++r) {
        if (row0 + r >= rows) break;
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(stage_at(base, r, at >> 2) + (at & 3) * 4) : "memory");
        if (keep) from_f32(v, keep[(row0 + r) * o.ld_keep[0] + c]);
        v = activate(v, o.act);
        if (add) v += to_f32(add[(row0 + r) * o.ld_add[p] + c]);
        from_f32(v, out[(row0 + r) * o.ld_out[p] + c]);
      }
    }
  }
  __syncwarp();
}

// out = act(g) * u of 32 rows x 64 columns: acc[0 .. 63] are g's sums, the others u's.  The other warp of the same
// rows (`half`) holds the other 64 columns of a group of 128.
template <typename T>
__device__ __forceinline__ void finish_gated(const RingParams& g, float (&acc)[128], uint8_t* stage, int lane, int quarter,
                                             int half, int64_t row0, int64_t col0, int64_t rows) {
  const FfnOut& o = g.o;
  const uint32_t base = smem_u32(stage);
  const int64_t cols = g.cols;
  if (o.codes[0].data) {
    if (col0 + 64 > cols) {   // (an infinity times a column that is not there is NaN)
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (col0 + i >= cols) acc[i] = acc[64 + i] = 0.f;
    }
    uint32_t mg = 0, mu = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      mg = max(mg, abs_bits(acc[i]));
      mu = max(mu, abs_bits(acc[64 + i]));
    }
    // the two warps that share the group show each other their maxima (both come here for every tile)
    const uint32_t mine = base + lane * 8, theirs = half ? mine - 4 * kRingWarpStage : mine + 4 * kRingWarpStage;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(mine), "r"(mg), "r"(mu) : "memory");
    asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
    uint32_t og, ou;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(og), "=r"(ou) : "r"(theirs) : "memory");
    asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
    const GroupScale sg = group_scale(max(mg, og), 448.f), su = group_scale(max(mu, ou), 448.f);
    if (row0 + lane < rows && col0 < cols) {
      if (half == 0) o.codes[0].scales[(row0 + lane) * o.codes[0].stride_row + (col0 >> 7) * o.codes[0].stride_col] = sg.scale;
      if (half == 0) o.codes[1].scales[(row0 + lane) * o.codes[1].stride_row + (col0 >> 7) * o.codes[1].stride_col] = su.scale;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float inv = i < 4 ? sg.inv : su.inv;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float* v = acc + 16 * i + 4 * j;
        w[j] = fp8x4<false>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      }
      st_shared_v4(base + sw128_offset(lane, i), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + lane / 8, c = lane % 8;
      uint4 v;
      ld_shared_v4(base + sw128_offset(r, c), v);
      const FfnCodes& q = o.codes[c >> 2];
      if (row0 + r < rows) store_codes16(q.data + (row0 + r) * q.ld, v, col0 + (c & 3) * 16, cols);
    }
  }
  const int lr = lane >> 3, lc = lane & 7;
  T* const out = static_cast<T*>(o.out[0]);
  T* const kg = static_cast<T*>(o.keep[0]);
  T* const ku = static_cast<T*>(o.keep[1]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float *x = acc + j * 32 + 4 * i, *y = x + 64;
      st_shared_v4(stage_at(base, lane, i), x[0], x[1], x[2], x[3]);
      st_shared_v4(stage_at(base, lane, 8 + i), y[0], y[1], y[2], y[3]);
    }
    __syncwarp();
    const int64_t first = col0 + j * 32;
    // eight lanes to a row, four columns each, where rows are on 16-byte boundaries
    const int64_t col = first + lc * 4;
    const bool mine = o.vec && col + 4 <= cols;
#pragma unroll 4
    for (int r = lr; r < 32; r += 4) {
      float v[4], u[4];
      ld_shared_v4(stage_at(base, r, lc), v[0], v[1], v[2], v[3]);
      ld_shared_v4(stage_at(base, r, 8 + lc), u[0], u[1], u[2], u[3]);
      if (!mine || row0 + r >= rows) continue;
      if (kg) {
        store_n(kg + (row0 + r) * o.ld_keep[0] + col, v);
        store_n(ku + (row0 + r) * o.ld_keep[1] + col, u);
      }
      activate_all(v, o.act);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= u[i];
      store_n(out + (row0 + r) * o.ld_out[0] + col, v);
    }
    // what is left of a row one by one, a lane to a column
    const int64_t rest = o.vec ? (cols & ~int64_t(3)) : 0, end = cols < first + 32 ? cols : first + 32;
    const int64_t c = (rest > first ? rest : first) + lane;
    if (c < end) {
      const int at = static_cast<int>(c - first);
#pragma unroll 4
      for (int r = 0; r < 32; ++r) {
        if (row0 + r >= rows) break;
        float v, u;
        const uint32_t in = (at & 3) * 4;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(stage_at(base, r, at >> 2) + in) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(stage_at(base, r, 8 + (at >> 2)) + in) : "memory");
        if (kg) {
          from_f32(v, kg[(row0 + r) * o.ld_keep[0] + c]);
          from_f32(u, ku[(row0 + r) * o.ld_keep[1] + c]);
        }
        from_f32(activate(v, o.act) * u, out[(row0 + r) * o.ld_out[0] + c]);
      }
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
// Maps: a of the first and second source or product, b likewise, or of the two weights of a gated product.
struct RingMaps {
  CUtensorMap a[2], b[2];
};

template <int BN, bool PAIR, bool GATED, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(RingShape<BN, PAIR>::THREADS, 1)
    ffn_ring_kernel(const __grid_constant__ RingMaps maps, const __grid_constant__ RingParams g) {
  using Sh = RingShape<BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + Sh::STAGES * Sh::STAGE;
  RingBarriers* bar = reinterpret_cast<RingBarriers*>(staging + Sh::EPI_WARPS * kRingWarpStage);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // (uniform for the compiler too)
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int worker = static_cast<int>(blockIdx.x) / Sh::CTAS;
  const int workers = static_cast<int>(gridDim.x) / Sh::CTAS;
  constexpr int TILE_COLS = GATED ? BN / 2 : BN;
  const int row_blocks = (g.rows + Sh::TILE_ROWS - 1) / Sh::TILE_ROWS;
  const int col_blocks = (g.cols + TILE_COLS - 1) / TILE_COLS;
  const int per_problem = row_blocks * col_blocks;
  const int tiles = per_problem * g.problems;
  const int kt = g.kt * g.sources;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Sh::STAGES; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->acc_full[a], 1);
      mbar_init(&bar->acc_empty[a], Sh::CTAS * Sh::EPI_WARPS);
    }
    mbar_init(&bar->drain, 1);
    bar->ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(&bar->tmem_base, Sh::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&bar->tmem_base, Sh::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_sync();   // both CTAs' barriers and TMEM exist before any signal between them
  else
    __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem = bar->tmem_base;
  CtaCtl* cta = &bar->ctl;
  int issued = 0, lost = -1;   // producer only: loads so far, and the one that the test hook skipped

  if (warp < 4) {
    if (Sh::SPLIT_REGS) regs_decrease<Sh::OTHER_REGS>();
    if (warp == 0 && lane == 0) {
      // ---------------- producer (every CTA) ----------------
      const int lose_tile = g.ctl.inject_lost_load ? tiles - 1 : -1;   // test hook: this tile's last load never comes
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = worker; ok && tile < tiles; tile += workers) {
        int rb, cb;
        const int problem = tile >= per_problem ? 1 : 0;
        ring_tile(tile - problem * per_problem, row_blocks, col_blocks, g.raster, rb, cb);
        const int a_row = rb * Sh::TILE_ROWS + static_cast<int>(rank) * Sh::A_ROWS;
        const int b_row = GATED ? cb * TILE_COLS : cb * BN + static_cast<int>(rank) * Sh::B_ROWS;
        for (int kb = 0; kb < kt; ++kb) {
          if (!mbar_wait(&bar->empty[s], ph ^ 1u, g.ctl, cta, kSiteProducerEmpty) || cta->abort) { ok = false; break; }
          const int second = kb >= g.kt ? 1 : 0;      // the second source
          const int k = (kb - second * g.kt) * kFfnBK;
          const CUtensorMap* ma = &maps.a[problem | second];
          const CUtensorMap* mb = &maps.b[GATED ? static_cast<int>(rank) : second];   // (two products share b)
          const uint32_t a_at = smem_u32(ring + s * Sh::STAGE), b_at = a_at + Sh::A_BYTES;
          auto load = [&](uint32_t at, const CUtensorMap* m, int x, int y) {
            if (PAIR)
              tma_load_2d_pair(at, m, mapa_shared(smem_u32(&bar->full[s]), 0), x, y);
            else
              tma_load_2d(at, m, &bar->full[s], x, y);
          };
          if (tile == lose_tile && kb == kt - 1) {
            lost = issued;
          } else {
            // (the even CTA's barrier counts the bytes of both CTAs' loads)
            if (rank == 0) mbar_arrive_expect_tx(&bar->full[s], Sh::CTAS * Sh::STAGE);
            if (A_MN) {
              load(a_at, ma, a_row, k);
              load(a_at + 8192, ma, a_row + 64, k);
            } else {
              load(a_at, ma, k, a_row);
            }
            if (B_MN) {
              load(b_at, mb, b_row, k);
              load(b_at + 8192, mb, b_row + 64, k);
            } else if (GATED && !PAIR) {
              load(b_at, mb, k, b_row);
              load(b_at + 8192, &maps.b[1], k, b_row);
            } else {
              load(b_at, mb, k, b_row);
            }
          }
          ++issued;
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (the even CTA of a pair) ----------------
      // The whole warp walks the loop, so that addresses and descriptors stay
      // in uniform registers; one lane issues.
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      const bool leader = ring_elect_one();
      const uint32_t ring0 = smem_u32(ring);
      const uint64_t a0 = A_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0);
      const uint64_t b0 = (B_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0)) + Sh::A_BYTES / 16;
      // 16 along K: 32 bytes of a K-major row, 16 rows of 128 bytes of an MN-major tile
      constexpr uint32_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;
      for (int tile = worker; ok && tile < tiles; tile += workers) {
        for (int kc = 0; ok && kc < kt; kc += g.restart) {
          const int end = min(kc + g.restart, kt);
          if (!__all_sync(0xffffffffu, mbar_wait(&bar->acc_empty[a], aph ^ 1u, g.ctl, cta, kSiteMmaAccEmpty))) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + a * BN;
          for (int kb = kc; kb < end; ++kb) {
            const bool there = mbar_wait(&bar->full[s], ph, g.ctl, cta, kSiteConsumerFull);
            tc_fence_after();
            const uint64_t da = a0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
            const uint64_t db = b0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
            if (leader && there) {   // (nothing of a slot that never came)
#pragma unroll
              for (int kk = 0; kk < kFfnBK / 16; ++kk) {
                const uint32_t more = kb > kc || kk > 0;
                if (PAIR)
                  umma_f16_pair(d, da + A_STEP * kk, db + B_STEP * kk, g.idesc, more);
                else
                  umma_f16(d, da + A_STEP * kk, db + B_STEP * kk, g.idesc, more);
              }
              if (PAIR) umma_commit_pair(&bar->empty[s], 0x3); else umma_commit(&bar->empty[s]);
            }
            // (the vote comes after the MMAs are issued, off their path)
            if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
            if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          if (leader) {
            if (PAIR) umma_commit_pair(&bar->acc_full[a], 0x3); else umma_commit(&bar->acc_full[a]);
          }
          if (++a == 2) { a = 0; aph ^= 1u; }
        }
      }
      if (leader) {
        // fires when every MMA issued above has completed
        if (PAIR) umma_commit_pair(&bar->drain, 0x1); else umma_commit(&bar->drain);
        CtaCtl never_abort{0};
        mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
      }
    }
  } else {
    // ---------------- outputs ----------------
    if (Sh::SPLIT_REGS) regs_increase<Sh::EPI_REGS>();
    const int e = warp - 4;
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int half = e >> 2;               // which half of the tile's columns
    uint8_t* my_stage = staging + e * kRingWarpStage;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // TMEM columns of a thread's sums 0 .. 63 and 64 .. 127
    const uint32_t lo = GATED ? half * 64 : half * 128, hi = GATED ? BN / 2 + half * 64 : half * 128 + 64;
    int a = 0;
    uint32_t aph = 0;
    bool ok = true;   // after a wait that gave up: nothing is written any more
    for (int tile = worker; tile < tiles; tile += workers) {
      int rb, cb;
      const int problem = tile >= per_problem ? 1 : 0;
      ring_tile(tile - problem * per_problem, row_blocks, col_blocks, g.raster, rb, cb);
      const int64_t row0 = static_cast<int64_t>(rb) * Sh::TILE_ROWS + rank * Sh::A_ROWS + quarter * 32;
      const int64_t col0 = static_cast<int64_t>(cb) * TILE_COLS + half * (GATED ? 64 : 128);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      if (!GATED && g.o.add[problem] && row0 + lane < g.rows) {
        // this thread's row of the addend comes into L2 while the products run
        const int size = g.o.out_f32 ? 4 : 2;
        const uint8_t* at = static_cast<const uint8_t*>(g.o.add[problem]) + ((row0 + lane) * g.o.ld_add[problem] + col0) * size;
#pragma unroll 1
        for (int i = 0; i < 128 && col0 + i < g.cols; i += 128 / size) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i * size));
      }
#pragma unroll 1
      for (int kc = 0; kc < kt; kc += g.restart) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bar->acc_full[a], aph, g.ctl, cta, kSiteEpilogueAccFull));
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + lanes + a * BN;
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(src + lo, v[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tmem_wait_ld();
          regs_after_wait(v[j & 1]);
          if (j < 3) {
            tmem_ld_32x32b_x32(src + (j + 1 < 2 ? lo + 32 : hi + (j - 1) * 32), v[(j + 1) & 1]);
          } else {
            // the buffer is in registers: hand it back to the MMA issuer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (PAIR)
                ring_arrive_cluster_relaxed(mapa_shared(smem_u32(&bar->acc_empty[a]), 0));
              else
                mbar_arrive(&bar->acc_empty[a]);
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[j * 32 + i] += __uint_as_float(v[j & 1][i]);
        }
        if (++a == 2) { a = 0; aph ^= 1u; }
      }
      const int64_t rows = ok ? g.rows : 0;
      if constexpr (GATED) {
        if (g.o.bf16)
          finish_gated<__nv_bfloat16>(g, acc, my_stage, lane, quarter, half, row0, col0, rows);
        else
          finish_gated<__half>(g, acc, my_stage, lane, quarter, half, row0, col0, rows);
      } else {
        if (g.o.bf16) {
          if (g.o.out_f32)
            finish_linear<__nv_bfloat16, float>(g, problem, acc, my_stage, lane, row0, col0, rows);
          else
            finish_linear<__nv_bfloat16, __nv_bfloat16>(g, problem, acc, my_stage, lane, row0, col0, rows);
        } else {
          if (g.o.out_f32)
            finish_linear<__half, float>(g, problem, acc, my_stage, lane, row0, col0, rows);
          else
            finish_linear<__half, __half>(g, problem, acc, my_stage, lane, row0, col0, rows);
        }
      }
    }
  }

  __syncthreads();
  if (cta->abort && warp == 0 && lane == 0) {
    if (PAIR) {
      // this CTA's loads count on the even CTA's barrier: give any still in
      // flight time to land before the pair tears down
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
    } else {
      // loads still in flight land in shared memory: wait for them before exit
      CtaCtl never_abort{0};
      for (int i = issued > Sh::STAGES ? issued - Sh::STAGES : 0; i < issued; ++i) {
        if (i == lost) continue;
        mbar_wait(&bar->full[i % Sh::STAGES], static_cast<uint32_t>((i / Sh::STAGES) & 1), g.ctl, &never_abort,
                  kSiteDrain);
      }
    }
  }
  if (PAIR) {
    tc_fence_before();
    cluster_sync();   // the even CTA's MMAs, which touch both CTAs, have completed
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, Sh::TMEM_COLS); else tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// Launch configuration of a kernel of `ctas` CTAs per cluster.
struct RingConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  RingConfig(int grid, int threads, int ctas, int smem, cudaStream_t stream) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (ctas > 1) {
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = ctas;
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
  }
};

inline CUtensorMapDataType ffn_map_type(const FfnOut& o) {
  return o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Map of an operand of `rows` x `summed`, stored summed axis first where `mn`, whose boxes hold box_rows of its rows.
inline cudaError_t ffn_map(CUtensorMap* m, const FfnProduct& p, const void* base, int64_t ld, int64_t rows, bool mn,
                           int box_rows) {
  const uint64_t row_bytes = static_cast<uint64_t>(ld) * 2;
  return mn ? make_tmap_2d(m, base, ffn_map_type(p.out), rows, p.summed, row_bytes, 64, kFfnBK, CU_TENSOR_MAP_SWIZZLE_128B)
            : make_tmap_2d(m, base, ffn_map_type(p.out), p.summed, rows, row_bytes, kFfnBK, box_rows,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

// With a register split, a kernel must have exactly kRingLaunchRegs at launch: with fewer, the increase would wait for ever.
inline cudaError_t check_launch_regs(std::atomic<int>& regs, const void* kernel) {
  if (regs.load() < 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs);
  }
  return regs.load() == kRingLaunchRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int BN, bool PAIR, bool GATED, bool A_MN, bool B_MN>
cudaError_t launch_ring(FfnProduct& p, const void** kernel) {
  using Sh = RingShape<BN, PAIR>;
  auto k = ffn_ring_kernel<BN, PAIR, GATED, A_MN, B_MN>;
  *kernel = reinterpret_cast<const void*>(k);
  const bool sum = p.op == kFfnInputGrad && p.count == 2, both = p.op == kFfnWeightGrad && p.count == 2;
  RingMaps maps = {};
  cudaError_t e;
  if (p.summed > 0) {
    const int b_box = GATED && !PAIR ? 64 : 128;
    if ((e = ffn_map(&maps.a[0], p, p.a[0], p.lda[0], p.rows, A_MN, 128)) != cudaSuccess) return e;
    if ((e = ffn_map(&maps.b[0], p, p.b[0], p.ldb[0], p.cols, B_MN, b_box)) != cudaSuccess) return e;
    if ((sum || both) && (e = ffn_map(&maps.a[1], p, p.a[1], p.lda[1], p.rows, A_MN, 128)) != cudaSuccess) return e;
    if ((sum || GATED) && (e = ffn_map(&maps.b[1], p, p.b[1], p.ldb[1], p.cols, B_MN, b_box)) != cudaSuccess) return e;
  }
  RingParams g = {};
  g.o = p.out;
  g.rows = static_cast<int32_t>(p.rows);
  g.cols = static_cast<int32_t>(p.cols);
  g.kt = static_cast<int32_t>((p.summed + kFfnBK - 1) / kFfnBK);
  g.sources = sum ? 2 : 1;
  g.problems = both ? 2 : 1;
  const bool wide = p.out.out_f32 || p.out.codes[0].data;
  g.restart = wide ? kFfnRestart : (g.kt > 0 ? g.kt * g.sources : 1);
  g.raster = p.plan.raster_gm;
  g.idesc = umma_idesc_f16(p.out.bf16 != 0, Sh::TILE_ROWS, BN) | (A_MN ? kIdescAMn : 0u) | (B_MN ? kIdescBMn : 0u);
  g.ctl = p.ctl;
  if (Sh::SPLIT_REGS) {
    static std::atomic<int> regs{-1};
    if ((e = check_launch_regs(regs, *kernel)) != cudaSuccess) return e;
  }
  if ((e = ensure_smem_attr(*kernel, Sh::SMEM)) != cudaSuccess) return e;
  RingConfig c(p.plan.grid, Sh::THREADS, Sh::CTAS, Sh::SMEM, p.stream);
  return cudaLaunchKernelEx(&c.cfg, k, maps, g);
}

}  // namespace gp
