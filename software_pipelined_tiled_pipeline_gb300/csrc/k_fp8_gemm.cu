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
//   warp 1      allocates TMEM and issues the MMAs of a K block into the next
//               TMEM buffer; their one commit both frees the ring slot and
//               hands the buffer to the adding warps
//   warps 4-11  bring the scales of 8 to 32 K blocks at a time into shared
//               memory (cp.async), add each TMEM buffer, scaled, to the sums in
//               their registers, and write C at a tile's end
// Warp w may read TMEM lanes 32 (w mod 4) .. +31; the two warps of a quarter
// take half the columns each.  "P" is the operand on the MMA's M side (128
// rows per CTA), "Q" the one on its N side (BN rows); either may be A.
//
// What bounds it: with every K block, 128 x BN sums change hands between the
// tensor cores and the adding warps (wait, TMEM read, FMA, release), about as
// long as the block's MMAs; no unit is near its limit alone.  Measured: 8192 x
// 8192 x 4096 (E4M3, row and block scales, BF16 out) 207 us, 2660 TFLOP/s, for
// some tens of calls in a row, as calls or in a graph, and 220 to 232 us where
// they go on for a second, as the power limit then takes the SM clock from 2070
// to 1870-1950 MHz; 186 us when the hand-over is left out.  4096 x 4096 x 8192
// with row scales on both sides 195 us, 227 with an FP32 addend.  For few rows
// the weights' bytes bound it: 1 x 8192 x 8192 15.3 us, 4.4 TB/s with its start
// and end.
#include <atomic>
#include <cstring>
#include "fp8_internal.h"
#include "gp_device.cuh"

namespace gp {
namespace {

constexpr int kBK = 128;                  // K block: bytes of a row per ring slot, and values per scale
constexpr int kMmaK = 32;                 // K of one kind::f8f6f4 instruction
constexpr int kThreads = 384;
constexpr int kAddWarps = 8;
constexpr int kAddThreads = 32 * kAddWarps;
constexpr int kStageWarpBytes = 32 * 128;   // output staging of one warp: 32 rows of 32 FP32
constexpr int kLaunchRegs = 168;          // registers per thread at launch, where warps trade them
constexpr int kMaxRing = 12;
constexpr int64_t kMaxTiles = int64_t(1) << 30;   // tile numbers plus a grid stay below 2^31

struct Fp8Barriers {
  uint64_t full[kMaxRing];
  uint64_t done[kMaxRing];   // the MMAs of the slot's K block have completed
  uint64_t acc_empty[4];
  uint64_t drain;
  uint32_t tmem_base;
  CtaCtl ctl;
};
constexpr int kFp8BarrierBytes = 256;
static_assert(sizeof(Fp8Barriers) <= kFp8BarrierBytes, "barrier region too small");

// PAIR: a cluster of two CTAs shares a 256 x BN tile, each holding 128 rows of
// P and BN / 2 of Q; one thread of the even CTA issues the MMAs (M = 256),
// which read both CTAs' halves and leave each its own 128 rows.
template <int BN, bool PAIR>
struct Fp8Shape {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int P_ROWS = 128;
  static constexpr int Q_ROWS = BN / CTAS;
  static constexpr int TILE_P = P_ROWS * CTAS;
  static constexpr int P_BYTES = P_ROWS * kBK;
  static constexpr int STAGE = (P_ROWS + Q_ROWS) * kBK;
  static constexpr int BUFS = BN == 256 ? 2 : 4;       // TMEM accumulators
  static constexpr uint32_t TMEM_COLS = BUFS * BN;
  static constexpr int HALF = BN / 2;                  // columns per adding warp
  static constexpr int SCALES = P_ROWS + BN;           // floats per K block: P's, then Q's
  // K blocks whose scales are staged together, in two batches in turn: as many
  // as cost no ring slot.  The code between two batches is cold each time it
  // comes: 8192 x 8192 x 4096 228 us with 8 together, 215 with 22, 207 with the 32
  // that 11 times a tile's scales hold; 4096 x 4096 x 8192 with row scales 206
  // with 8, 190 with 16.  (Three batches of 5 and 8
  // with a barrier that nobody waits for: 223 and 202.)
  static constexpr int BATCH = BN == 256 ? 11 : (BN >= 64 ? 16 : 8);
  static constexpr int FIXED = kAddWarps * kStageWarpBytes + 2 * BATCH * SCALES * 4 + kFp8BarrierBytes + 1024;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kMaxRing ? FIT : kMaxRing;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  // A slot's barrier tells the adding warps one phase from the next only while
  // the MMAs cannot be a whole ring ahead of them.
  static_assert(BUFS < STAGES, "more accumulators than ring slots");
  // The adding warps of a wide tile hold its sums in registers, and take them
  // from the other four warps: ADD_REGS and OTHER_REGS per thread.
  static constexpr bool SPLIT_REGS = BN >= 128;
  static constexpr int ADD_REGS = BN == 256 ? 216 : 208, OTHER_REGS = BN == 256 ? 72 : 88;
  static_assert(kThreads * kLaunchRegs == 32 * (kAddWarps * ADD_REGS + (kThreads / 32 - kAddWarps) * OTHER_REGS),
                "register split");
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
  int32_t vec16;             // groups of 8 16-bit outputs are aligned to 16 bytes
  uint32_t idesc;
  int32_t raster_gp;         // P blocks per raster group
  int32_t k_log;             // log2 of the CTAs (one cluster) that share a tile's K blocks; one tile per cluster then
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

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
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

// Arrive on an mbarrier of another CTA of the cluster without ordering memory:
// the TMEM buffer it hands back has been read into registers, and nothing else
// is handed over.  (The releasing form waits for this warp's earlier stores
// with every K block.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Store 4 bytes into another CTA's shared memory (cluster-window address).
__device__ __forceinline__ void st_cluster_s32(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f1(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// 4 bytes from global to shared memory without a register; zeros where !valid (nothing is read then).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Waits that come with every K block.  The try itself waits in hardware, up to
// kTryNs; the clock is read only where that is not enough.  One that gives up
// leaves its site in the CTA's abort flag, which is reported when the kernel
// ends and makes every further wait return after two tries: the producer and
// the MMA issuer leave their loops at that, the adding warps after at most a
// batch of K blocks (7 ms).  Code and registers here are counted, as the K loop
// of the adding warps fills both.
constexpr uint32_t kTryNs = 100000;
constexpr uint64_t kMostWaitNs = 4000000000ull;   // the 32-bit clock wraps after 4.29 s
__device__ __forceinline__ bool try_wait(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity), "n"(kTryNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t clock_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool ring_wait(uint32_t bar_addr, uint32_t parity, uint32_t limit_ns, CtaCtl* cta,
                                          int site) {
  if (try_wait(bar_addr, parity)) return true;
  const uint32_t t0 = clock_ns();
  while (!try_wait(bar_addr, parity)) {
    if (cta->abort) return false;
    if (clock_ns() - t0 > limit_ns) {
      cta->abort = site;
      return false;
    }
  }
  return true;
}

// Pairs of FP32 values in one 64-bit register: a packed product is one
// instruction, and rounds each half as a single one does.  (Packed FMAs on what
// the TMEM loads return cost as many moves as they save.)
__device__ __forceinline__ uint64_t pack2f(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Output tile -> its P and Q blocks: groups of `gp` P blocks, each swept over all Q blocks, so that the
// CTAs at work at one time share operands in L2.
__device__ __forceinline__ void tile_blocks(int tile, int p_blocks, int q_blocks, int gp, int& pb, int& qb) {
  const int per = gp * q_blocks;
  const int group = tile / per;
  const int first = group * gp;
  const int n = min(gp, p_blocks - first);
  const int in = tile - group * per;
  pb = first + in % n;
  qb = in / n;
}

// The work of one worker (a CTA, a pair, or a cluster that splits the K loop),
// walked alike by all its warps: every `step`-th tile, K blocks k0 .. k1 - 1.
struct Items {
  int tile, tiles, step, k0, k1;
  __device__ __forceinline__ bool next() {
    tile += step;
    return tile < tiles;
  }
};

__device__ __forceinline__ void add_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kAddThreads) : "memory"); }

template <typename T>
__device__ __forceinline__ float widen(T t) { return static_cast<float>(t); }
template <typename T>
__device__ __forceinline__ T narrow(float f) { return static_cast<T>(f); }   // nearest even
template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T e[4];
};

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  const T v[2] = {narrow<T>(lo), narrow<T>(hi)};
  uint32_t r;
  memcpy(&r, v, 4);
  return r;
}

// Write a warp's 32 rows x HALF columns of sums (thread: one row) to C: through
// shared memory, so that a row's outputs leave side by side.  16-byte chunk c
// of row r of the staged 32 x 128 bytes lies at c ^ (r mod 8).
template <int HALF, bool ADD, typename T>
__device__ __forceinline__ void write_out(const Fp8Params& g, const float (&acc)[HALF], uint8_t* stage, int lane,
                                          int64_t p0, int64_t q0) {
  T* const c = static_cast<T*>(g.c);
  const T* const add = ADD ? static_cast<const T*>(g.addend) : nullptr;
  if (g.swapped) {
    // The lanes' rows are C's columns: each of C's rows gets 32 neighbouring
    // outputs.  Sums go through shared memory (each lane reads back its own) so
    // that the loop over them is short code: a cold instruction costs more than
    // the round trip.
    constexpr int CW = HALF < 32 ? HALF : 32;
    const int64_t col = p0 + lane;
    float* mine = reinterpret_cast<float*>(stage) + lane;
#pragma unroll
    for (int j = 0; j < HALF / CW; ++j) {
#pragma unroll
      for (int i = 0; i < CW; ++i) mine[i * 32] = acc[j * CW + i];
      const int64_t first = q0 + j * CW, left = g.q.rows - first;
      const int rows = col < g.p.rows ? static_cast<int>(left < CW ? left : CW) : 0;
      T* o = c + first * g.ldc + col;
      const T* f = ADD ? add + first * g.ld_add + col : nullptr;
#pragma unroll 1
      for (int i = 0; i < rows; ++i, o += g.ldc) {
        float v = mine[i * 32];
        if (ADD) {
          v += widen(*f);
          f += g.ld_add;
        }
        *o = narrow<T>(v);
      }
    }
    return;
  }
  const uint32_t base = smem_u32(stage);
  const bool full = g.vec && p0 + 32 <= g.p.rows && q0 + HALF <= g.q.rows;
  if constexpr (sizeof(T) == 2 && HALF >= 64) {
    if (!ADD && full && g.vec16) {
      // 64 columns at a time, rounded before they are staged: 16 bytes per lane, 8 lanes per row
      T* out = c + (p0 + lane / 8) * g.ldc + q0 + lane % 8 * 8;
#pragma unroll
      for (int j = 0; j < HALF / 64; ++j, out += 64) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* x = acc + j * 64 + 8 * i;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + sw128_offset(lane, i)),
                       "r"(pack16<T>(x[0], x[1])), "r"(pack16<T>(x[2], x[3])), "r"(pack16<T>(x[4], x[5])),
                       "r"(pack16<T>(x[6], x[7]))
                       : "memory");
        }
        __syncwarp();
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                       : "r"(base + sw128_offset(i * 4 + lane / 8, lane % 8))
                       : "memory");
        T* o = out;
#pragma unroll
        for (int i = 0; i < 8; ++i, o += 4 * g.ldc) *reinterpret_cast<uint4*>(o) = w[i];
      }
      return;
    }
  }
  constexpr int CW = HALF < 32 ? HALF : 32;      // columns staged at a time, in FP32
  constexpr int PER = CW / 4;                    // lanes per row when they leave
  const int64_t row = p0 + lane / PER, col = q0 + lane % PER * 4;
  T* out = c + row * g.ldc + col;
  const T* from = ADD ? add + row * g.ld_add + col : nullptr;
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
    if (!full) {
      // A tile that C ends in, or whose rows are off their alignment: one
      // output per lane, CW lanes to a row, eight steps' addends at a time.
      constexpr int AT_ONCE = 32 / CW;             // rows per step
      const int cl = lane % CW, rl = lane / CW;
      const int64_t q = q0 + j * CW + cl;
      const int rows = q < g.q.rows ? static_cast<int>(g.p.rows - p0 < 32 ? g.p.rows - p0 : 32) : 0;   // (may be < 0)
      const uint32_t from_col = static_cast<uint32_t>(cl / 4);
#pragma unroll 1
      for (int r0 = rl; r0 < rows; r0 += 8 * AT_ONCE) {
        T* o = c + (p0 + r0) * g.ldc + q;
        T was[8];
        if (ADD) {
          const T* f = add + (p0 + r0) * g.ld_add + q;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (r0 + u * AT_ONCE < rows) was[u] = f[u * AT_ONCE * g.ld_add];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = r0 + u * AT_ONCE;
          if (r < rows) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(base + sw128_offset(r, from_col) + cl % 4 * 4) : "memory");
            o[u * AT_ONCE * g.ldc] = narrow<T>(ADD ? v + widen(was[u]) : v);
          }
        }
      }
      continue;
    }
    // Addends are asked for four rows' worth at a time before the first of
    // these outputs is written: they may be the same memory.
    constexpr int GROUP = ADD && PER > 4 ? 4 : PER;
#pragma unroll
    for (int i0 = 0; i0 < PER; i0 += GROUP) {
      Four<T> was[GROUP];
      if (ADD) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
          was[i] = *reinterpret_cast<const Four<T>*>(from + (i0 + i) * (32 / PER) * g.ld_add + j * CW);
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(base + sw128_offset((i0 + i) * (32 / PER) + lane / PER, lane % PER))
                     : "memory");
        Four<T> o;
        o.e[0] = narrow<T>(ADD ? v.x + widen(was[i].e[0]) : v.x);
        o.e[1] = narrow<T>(ADD ? v.y + widen(was[i].e[1]) : v.y);
        o.e[2] = narrow<T>(ADD ? v.z + widen(was[i].e[2]) : v.z);
        o.e[3] = narrow<T>(ADD ? v.w + widen(was[i].e[3]) : v.w);
        *reinterpret_cast<Four<T>*>(out + (i0 + i) * (32 / PER) * g.ldc + j * CW) = o;
      }
    }
  }
}

// The K loop split over a cluster: every CTA hands each of the others the
// columns that are theirs, and writes its own.  Buffer of a CTA: for each
// source, its columns of kXRow floats, one per row and one to keep the lanes of
// either walk off each other's banks.
constexpr int kXRow = 129;
template <bool ADD, typename T>
__device__ __forceinline__ void write_shared(const Fp8Params& g, const float* buf, int t, int ctas, int per_log,
                                             int64_t p0, int64_t q0) {
  T* const c = static_cast<T*>(g.c);
  const T* const add = ADD ? static_cast<const T*>(g.addend) : nullptr;
#pragma unroll 4
  for (int i = t; i < 128 << per_log; i += kAddThreads) {
    // neighbouring lanes along a row of C
    const int col = g.swapped ? i >> 7 : i & ((1 << per_log) - 1);
    const int row = g.swapped ? i & 127 : i >> per_log;
    float v = 0.f;       // in K order
    for (int s = 0; s < ctas; ++s) v += buf[((s << per_log) + col) * kXRow + row];
    const int64_t p = p0 + row, q = q0 + col;
    if (p >= g.p.rows || q >= g.q.rows) continue;
    const int64_t m = g.swapped ? q : p, n = g.swapped ? p : q;
    if (ADD) v += widen(add[m * g.ld_add + n]);
    c[m * g.ldc + n] = narrow<T>(v);
  }
}

// QROWS: Q has a scale for each row (a column of the tile); else one for each 128 rows.  ADD: there is an addend.
template <int BN, bool QROWS, bool PAIR, bool ADD>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_ring_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ Fp8Params g) {
  using Sh = Fp8Shape<BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + Sh::STAGES * Sh::STAGE;
  float* scales = reinterpret_cast<float*>(staging + kAddWarps * kStageWarpBytes);
  Fp8Barriers* bar = reinterpret_cast<Fp8Barriers*>(scales + 2 * Sh::BATCH * Sh::SCALES);

  // K blocks whose scales are staged together; with one scale for 128 of Q's rows the same memory holds more.
  constexpr int SCALES = QROWS ? Sh::SCALES : Sh::P_ROWS + 4;
  constexpr int BATCH = Sh::BATCH * Sh::SCALES / SCALES;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // (uniform for the compiler too)
  const int lane = threadIdx.x & 31;
  const int k_ctas = PAIR ? 1 : 1 << g.k_log;                 // CTAs that share a tile's K blocks
  const uint32_t in_cluster = PAIR || k_ctas > 1 ? cluster_ctarank() : 0u;
  const uint32_t rank = PAIR ? in_cluster : 0u;               // in the pair
  const int per_worker = Sh::CTAS * k_ctas;
  const int worker = static_cast<int>(blockIdx.x) / per_worker;
  const int workers = static_cast<int>(gridDim.x) / per_worker;
  const int p_blocks = (g.p.rows + Sh::TILE_P - 1) / Sh::TILE_P;
  const int q_blocks = (g.q.rows + BN - 1) / BN;
  const int kt = (g.K + kBK - 1) / kBK;
  Items items{worker - workers, p_blocks * q_blocks, workers, 0, kt};
  if (!PAIR && k_ctas > 1) {
    items.k0 = static_cast<int>((static_cast<int64_t>(kt) * in_cluster) >> g.k_log);
    items.k1 = static_cast<int>((static_cast<int64_t>(kt) * (in_cluster + 1)) >> g.k_log);
  }
  const int k0 = items.k0, k1 = items.k1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Sh::STAGES; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->done[s], 1);
    }
    for (int a = 0; a < Sh::BUFS; ++a) mbar_init(&bar->acc_empty[a], Sh::CTAS * kAddWarps);
    mbar_init(&bar->drain, 1);
    bar->ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
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
  // While the work before this kernel finishes, its first boxes come into L2:
  // a prefetch writes nothing, and L2 stays coherent with what is still written.
  if (warp == 0 && lane == 0 && worker < items.tiles) {
    int pb, qb;
    tile_blocks(worker, p_blocks, q_blocks, g.raster_gp, pb, qb);
    for (int kb = k0; kb < k1 && kb < k0 + Sh::STAGES; ++kb) {
      tma_prefetch_l2_2d(&tmP, kb * kBK, pb * Sh::TILE_P + rank * Sh::P_ROWS);
      tma_prefetch_l2_2d(&tmQ, kb * kBK, qb * BN + rank * Sh::Q_ROWS);
    }
  }
  pdl_wait();
  const uint32_t tmem = bar->tmem_base;
  CtaCtl* cta = &bar->ctl;
  const uint32_t limit_ns = static_cast<uint32_t>(g.ctl.timeout_ns < kMostWaitNs ? g.ctl.timeout_ns : kMostWaitNs);
  const uint32_t full0 = smem_u32(&bar->full[0]), done0 = smem_u32(&bar->done[0]), free0 = smem_u32(&bar->acc_empty[0]);
  int issued = 0, lost = -1;   // producer only: loads so far, and the one that the test hook skipped

  if (warp < 4) {
    if (Sh::SPLIT_REGS) regs_decrease<Sh::OTHER_REGS>();
    if (warp == 0 && lane == 0) {
      // ---------------- producer (every CTA) ----------------
      const int lose = g.ctl.inject_lost_load;   // test hook: the load of this tile and K block never comes
      const int lose_tile = lose == 0 ? -1 : (lose == 2 ? 0 : items.tiles - 1), lose_kb = lose == 2 ? 0 : kt - 1;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && items.next()) {
        int pb, qb;
        tile_blocks(items.tile, p_blocks, q_blocks, g.raster_gp, pb, qb);
        const int p_row = pb * Sh::TILE_P + rank * Sh::P_ROWS;
        const int q_row = qb * BN + rank * Sh::Q_ROWS;
        for (int kb = k0; kb < k1; ++kb) {
          if (!ring_wait(done0 + s * 8, ph ^ 1u, limit_ns, cta, kSiteProducerEmpty) || cta->abort) { ok = false; break; }
          uint8_t* slot = ring + s * Sh::STAGE;
          if (PAIR) {
            // the even CTA's barrier counts the bytes of both CTAs' loads
            if (rank == 0) mbar_arrive_expect_tx(&bar->full[s], 2 * Sh::STAGE);
            const uint32_t full = mapa_shared(smem_u32(&bar->full[s]), 0);
            tma_load_2d_pair(smem_u32(slot), &tmP, full, kb * kBK, p_row);
            tma_load_2d_pair(smem_u32(slot + Sh::P_BYTES), &tmQ, full, kb * kBK, q_row);
          } else if (items.tile != lose_tile || kb != lose_kb) {
            mbar_arrive_expect_tx(&bar->full[s], Sh::STAGE);
            tma_load_2d(smem_u32(slot), &tmP, &bar->full[s], kb * kBK, p_row);
            tma_load_2d(smem_u32(slot + Sh::P_BYTES), &tmQ, &bar->full[s], kb * kBK, q_row);
          } else {
            lost = issued;
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
      const bool leader = elect_one();
      const uint64_t desc0 = umma_desc_sw128(smem_u32(ring));
      while (ok && items.next()) {
        for (int kb = k0; kb < k1; ++kb) {
          const bool there = ring_wait(full0 + s * 8, ph, limit_ns, cta, kSiteConsumerFull) &&
                             ring_wait(free0 + a * 8, aph ^ 1u, limit_ns, cta, kSiteMmaAccEmpty);
          tc_fence_after();
          const uint64_t dp = desc0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
          const uint64_t dq = dp + Sh::P_BYTES / 16;
          const uint32_t d = tmem + a * BN;
          if (leader && there) {   // (nothing of a slot that never came, in a pair for neither CTA)
#pragma unroll
            for (int kk = 0; kk < kBK / kMmaK; ++kk) {   // 32 bytes along K: the start address field moves by 2
              if (PAIR)
                umma_f8_pair(d, dp + 2 * kk, dq + 2 * kk, g.idesc, kk == 0 ? 0u : 1u);
              else
                umma_f8(d, dp + 2 * kk, dq + 2 * kk, g.idesc, kk == 0 ? 0u : 1u);
            }
            if (PAIR) umma_commit_pair(&bar->done[s], 0x3); else umma_commit(&bar->done[s]);
          }
          // (the vote comes after the MMAs are issued, off their path)
          if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
          if (++a == Sh::BUFS) { a = 0; aph ^= 1u; }
        }
      }
      if (leader) {
        // fires when every MMA issued above has completed
        if (PAIR) umma_commit_pair(&bar->drain, 0x1); else umma_commit(&bar->drain);
        CtaCtl never_abort{0};
        mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
      }
    }
    if (!PAIR && k_ctas > 1 && worker < items.tiles) {
      // the adding warps' two barriers around their exchange (below); between
      // them a CTA that gave up tells the others, so that none of them writes
      // what its sums are missing from
      __syncwarp();
      cluster_sync();
      if (warp == 2 && lane < k_ctas && cta->abort)
        st_cluster_s32(mapa_shared(smem_u32(const_cast<int*>(&cta->abort)), lane), kSiteEpilogueAccFull);
      __syncwarp();
      cluster_sync();
    }
  } else {
    // ---------------- scaled sums and output ----------------
    if (Sh::SPLIT_REGS) regs_increase<Sh::ADD_REGS>();
    const int e = warp - 4;
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int half = e >> 2;               // which half of the columns
    const int row = quarter * 32 + lane;   // row of the CTA's tile that this thread holds
    uint8_t* my_stage = staging + e * kStageWarpBytes;
    constexpr int CW = Sh::HALF < 32 ? Sh::HALF : 32;
    constexpr int CHUNKS = Sh::HALF / CW;
    constexpr int LOG_BN = BN == 256 ? 8 : BN == 128 ? 7 : BN == 64 ? 6 : BN == 32 ? 5 : 4;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int s = 0, a = 0, batch = 0;
    uint32_t ph = 0;
    const int t = threadIdx.x - 128;
    const uint32_t lead_free0 = PAIR ? mapa_shared(free0, 0) : free0;
    bool ok = true;   // after a wait that gave up: no more data, but the barriers go on

    // Scales of K blocks kb .. of the tile (pb, qb) into staging batch `to`:
    // one per row, or one per 128 rows where that is all there is.
    const int p_log = g.p.shift ? 0 : 7;                                   // log2 of P's values per K block
    constexpr int Q_LOG = QROWS ? LOG_BN : (BN == 256 ? 1 : 0);
    auto stage_scales = [&](int to, int pb, int qb, int kb, int n) {
      const uint32_t slot = smem_u32(scales + to * BATCH * SCALES);
      auto one = [&](const ScaleView& v, int64_t first, int log, int step, int at) {
        // (a thread's values lie in one row: their addresses differ by a stride)
        const int r = t & ((1 << log) - 1), b0 = t >> log, by = kAddThreads >> log;
        const int64_t row = first + r * step;
        const bool in = row < v.rows;
        const float* from = v.base + (in ? (row >> v.shift) * v.stride_row + (kb + b0) * v.stride_col : 0);
        const int64_t next = in ? by * v.stride_col : 0;
        uint32_t dst = slot + (b0 * SCALES + at + r) * 4;
        for (int b = b0; b < n; b += by, from += next, dst += by * (SCALES * 4)) cp_async4(dst, from, in);
      };
      one(g.p, static_cast<int64_t>(pb) * Sh::TILE_P + rank * Sh::P_ROWS, p_log, 1, 0);
      one(g.q, static_cast<int64_t>(qb) * BN, Q_LOG, QROWS ? 1 : 128, Sh::P_ROWS);
    };
    while (items.next()) {
      float acc[Sh::HALF];
#pragma unroll
      for (int i = 0; i < Sh::HALF; ++i) acc[i] = 0.f;
      int pb, qb;
      tile_blocks(items.tile, p_blocks, q_blocks, g.raster_gp, pb, qb);
      if (ok && items.tile == worker) stage_scales(batch, pb, qb, k0, min(BATCH, k1 - k0));
      if (ADD && !g.swapped) {
        // this thread's row of the addend comes into L2 while the K loop runs
        const int size = g.out_type == GP_REAL_F32 ? 4 : 2;
        const int64_t p = static_cast<int64_t>(pb) * Sh::TILE_P + rank * Sh::P_ROWS + row;
        const int64_t q = static_cast<int64_t>(qb) * BN + half * Sh::HALF;
        if (p < g.p.rows) {
          const uint8_t* at = static_cast<const uint8_t*>(g.addend) + (p * g.ld_add + q) * size;
#pragma unroll 1
          for (int i = 0; i < Sh::HALF && q + i < g.q.rows; i += 128 / size)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i * size));
        }
      }
      for (int kc = k0; kc < k1; kc += BATCH, batch ^= 1) {
        const int end = min(kc + BATCH, k1);
        cp_async_wait_all();
        add_warps_sync();      // this batch is there for all, and all have read the one before
        if (!ok) continue;
        if (end < k1) stage_scales(batch ^ 1, pb, qb, end, min(BATCH, k1 - end));
        const float* slot = scales + batch * BATCH * SCALES;
        // A wait that gave up in here leaves wrong sums behind, which are never
        // written: the abort flag is looked at after each batch, and the CTAs of
        // a cluster tell each other.
        for (int kb = kc; kb < end; ++kb, slot += SCALES) {
          const float sp = slot[g.p.shift ? 0 : row];
          const float* sq = slot + Sh::P_ROWS;
          const float one = QROWS ? sp : sp * sq[BN == 256 ? half : 0];
          ring_wait(done0 + s * 8, ph, limit_ns, cta, kSiteEpilogueAccFull);
          __syncwarp();
          tc_fence_after();
          const uint32_t src = tmem + lanes + a * BN + half * Sh::HALF;
          uint32_t v[2][CW];
          tmem_ld(src, v[0]);
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) {
            tmem_wait_ld();
            regs_after_wait(v[j & 1]);
            if (j + 1 < CHUNKS) {
              tmem_ld(src + (j + 1) * CW, v[(j + 1) & 1]);
            } else {
              // the buffer is in registers: hand it back to the MMA issuer
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (PAIR)
                  mbar_arrive_cluster_relaxed(lead_free0 + a * 8);
                else
                  mbar_arrive(&bar->acc_empty[a]);
              }
            }
            float* o = acc + j * CW;
            const uint32_t* d = v[j & 1];
            if (QROWS) {
              const ulonglong2* q4 = reinterpret_cast<const ulonglong2*>(sq + half * Sh::HALF + j * CW);
              const uint64_t sp2 = pack2f(one, one);
#pragma unroll
              for (int i = 0; i < CW / 4; ++i) {
                const ulonglong2 q = q4[i];      // four columns' scales
                const uint64_t m = mul2(sp2, q.x), n = mul2(sp2, q.y);
                o[4 * i] = fmaf(__uint_as_float(d[4 * i]), lo2(m), o[4 * i]);
                o[4 * i + 1] = fmaf(__uint_as_float(d[4 * i + 1]), hi2(m), o[4 * i + 1]);
                o[4 * i + 2] = fmaf(__uint_as_float(d[4 * i + 2]), lo2(n), o[4 * i + 2]);
                o[4 * i + 3] = fmaf(__uint_as_float(d[4 * i + 3]), hi2(n), o[4 * i + 3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < CW; ++i) o[i] = fmaf(__uint_as_float(d[i]), one, o[i]);
            }
          }
          if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
          if (++a == Sh::BUFS) a = 0;
        }
        if (__any_sync(0xffffffffu, cta->abort)) ok = false;
      }
      if (!PAIR && k_ctas > 1) {
        // The ring has served its last K block, in every CTA of the cluster
        // after this: its memory takes the others' sums.
        cluster_sync();
        const int per_log = LOG_BN - g.k_log, per = 1 << per_log;    // columns per CTA
        const uint32_t at = smem_u32(ring) + ((in_cluster << per_log) * kXRow + row) * 4;
#pragma unroll
        for (int i = 0; i < Sh::HALF; ++i) {
          const int col = half * Sh::HALF + i;
          st_cluster_f1(mapa_shared(at + (col & (per - 1)) * (kXRow * 4), static_cast<uint32_t>(col >> per_log)), acc[i]);
        }
        cluster_sync();
        if (!cta->abort) {
          const float* buf = reinterpret_cast<const float*>(ring);
          const int64_t p0 = static_cast<int64_t>(pb) * Sh::TILE_P, q0 = static_cast<int64_t>(qb) * BN + in_cluster * per;
          if (g.out_type == GP_REAL_BF16)
            write_shared<ADD, __nv_bfloat16>(g, buf, t, k_ctas, per_log, p0, q0);
          else if (g.out_type == GP_REAL_F16)
            write_shared<ADD, __half>(g, buf, t, k_ctas, per_log, p0, q0);
          else
            write_shared<ADD, float>(g, buf, t, k_ctas, per_log, p0, q0);
        }
        continue;
      }
      if (!ok) continue;
      if (items.tile + items.step < items.tiles) {
        // the next tile's first scales come while this one is written
        int pn, qn;
        tile_blocks(items.tile + items.step, p_blocks, q_blocks, g.raster_gp, pn, qn);
        stage_scales(batch, pn, qn, k0, min(BATCH, k1 - k0));
      }
      const int64_t p0 = static_cast<int64_t>(pb) * Sh::TILE_P + rank * Sh::P_ROWS + quarter * 32;
      const int64_t q0 = static_cast<int64_t>(qb) * BN + half * Sh::HALF;
      if (g.out_type == GP_REAL_BF16)
        write_out<Sh::HALF, ADD, __nv_bfloat16>(g, acc, my_stage, lane, p0, q0);
      else if (g.out_type == GP_REAL_F16)
        write_out<Sh::HALF, ADD, __half>(g, acc, my_stage, lane, p0, q0);
      else
        write_out<Sh::HALF, ADD, float>(g, acc, my_stage, lane, p0, q0);
    }
  }

  __syncthreads();
  if (cta->abort && warp == 0 && lane == 0) {
    report_error(g.ctl, kDevErrTimeout, static_cast<uint32_t>(cta->abort));
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

// Launch configuration of a kernel of CTAS CTAs per cluster.
struct Config {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Config(int grid, int ctas, int smem, cudaStream_t stream) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
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

template <int BN, bool QROWS, bool PAIR, bool ADD>
cudaError_t launch_as(Fp8GemmArgs& a, const void** kernel) {
  using Sh = Fp8Shape<BN, PAIR>;
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
  const int size = real_bytes(a.out_type);
  auto aligned = [&](const void* p, int64_t ld, int64_t to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && ld * size % to == 0;
  };
  g.vec = aligned(a.C, a.ldc, 4 * size) && (!a.addend || aligned(a.addend, a.ld_add, 4 * size));
  g.vec16 = size == 2 && aligned(a.C, a.ldc, 16);
  g.idesc = idesc_f8(P.format, Q.format, Sh::TILE_P, BN);
  g.raster_gp = a.plan.raster_gm;
  g.k_log = a.plan.k_splits == 8 ? 3 : (a.plan.k_splits == 4 ? 2 : (a.plan.k_splits == 2 ? 1 : 0));
  g.ctl = a.ctl;
  auto k = fp8_ring_kernel<BN, QROWS, PAIR, ADD>;
  *kernel = reinterpret_cast<const void*>(k);
  if (Sh::SPLIT_REGS) {
    // The register split counts on exactly kLaunchRegs per thread at launch:
    // with fewer, the increase would wait for ever.  Refuse such a build.
    static std::atomic<int> regs{-1};
    if (regs.load() < 0) {
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
      regs.store(fa.numRegs);
    }
    if (regs.load() != kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  if ((e = ensure_smem_attr(*kernel, Sh::SMEM)) != cudaSuccess) return e;
  Config c(a.plan.grid, Sh::CTAS * a.plan.k_splits, Sh::SMEM, a.stream);
  return cudaLaunchKernelEx(&c.cfg, k, tmP, tmQ, g);
}

template <int BN, bool QROWS, bool PAIR>
cudaError_t launch_ring(Fp8GemmArgs& a, const void** kernel) {
  return a.addend ? launch_as<BN, QROWS, PAIR, true>(a, kernel) : launch_as<BN, QROWS, PAIR, false>(a, kernel);
}

template <int BN, bool PAIR>
void shape_of(gp_plan* p) {
  using Sh = Fp8Shape<BN, PAIR>;
  p->cta_pair = PAIR;
  p->bm = Sh::TILE_P;
  p->bn = BN;
  p->bk = kBK;
  p->stages = Sh::STAGES;
  p->stage_bytes = Sh::STAGE;
  p->ring_bytes = Sh::STAGES * Sh::STAGE;
  p->smem_bytes = Sh::SMEM;
  p->tmem_cols = Sh::TMEM_COLS;
}

// Pairs that fit on the device at once (cached per device).
cudaError_t pair_capacity(int* pairs) {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && (*pairs = cached[dev].load()) > 0) return cudaSuccess;
  using Sh = Fp8Shape<256, true>;
  const void* k = reinterpret_cast<const void*>(fp8_ring_kernel<256, false, true, false>);
  if ((e = ensure_smem_attr(k, Sh::SMEM)) != cudaSuccess) return e;
  Config c(2, 2, Sh::SMEM, nullptr);
  if ((e = cudaOccupancyMaxActiveClusters(pairs, k, &c.cfg)) != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorLaunchOutOfResources;
  if (dev >= 0 && dev < 64) cached[dev].store(*pairs);
  return cudaSuccess;
}

}  // namespace

namespace {

// What the planner knows of a tile width, in ns, measured on a 152-SM GB300
// (device time of whole calls in a graph, operands from HBM): a K block with Q
// block-scaled and row-scaled, the call around one tile per CTA, each further
// tile, and the exchange where a cluster splits the K loop.  For example, unsplit
// against two CTAs per tile: 48 x 8192 x 8192 25.6 -> 19.2 us (BN 64), 256 x
// 4096 x 4096 14.0 -> 20.0 us (BN 128); BN 64 against 128 at 1000 x 776 x 2056
// 9.8 and 10.1 us, BN 128 against 256 at 1024 x 4096 x 4096 25.5 and 18.3 us and
// at 512 x 4096 x 4096 14.6 and 16.7 us.
struct TileCost {
  int bn, k_block, k_rows, call, more, exchange;
};
constexpr TileCost kTileCosts[] = {{16, 255, 255, 3200, 300, 800},
                                   {32, 285, 285, 3500, 400, 1200},
                                   {64, 350, 350, 4200, 600, 2000},
                                   {128, 315, 395, 5000, 1000, 8000},
                                   {256, 385, 750, 6500, 1800, 0}};
constexpr double kReadGbs = 6500;        // operands from HBM
constexpr int kSwappedNs = 13;           // a column of a swapped tile's epilogue
constexpr int kMinShare = 4;             // K blocks of each CTA of a cluster, at least

}  // namespace

int fp8_plan_impl(int64_t M, int64_t N, int64_t K, int a_group, int b_group, int sms, const gp_fp8_options* opts,
                  gp_plan* p) {
  std::memset(p, 0, sizeof(*p));
  const int want = opts ? opts->bn : 0;
  bool known = want == 0;
  for (const TileCost& t : kTileCosts) known |= t.bn == want;
  if (!known) return GP_ERR_UNSUPPORTED;
  const bool no_pair = opts && opts->inject_lost_load;   // (a lost load is not injected into pairs)
  if (no_pair && want == 256) return GP_ERR_UNSUPPORTED;
  const int64_t kt = (K + kBK - 1) / kBK;
  const int have = sms > 0 ? sms : 152;
  // Try every width with either operand on the MMA's N side (Q), and every
  // cluster that keeps all of its tiles resident (clusters of 4 and 8 cannot
  // use every SM); take the least estimate.
  double best = 0;
  const TileCost* tile = nullptr;
  int best_c = 1;
  bool swapped = false;
  for (int sw = 0; sw < 2; ++sw) {
    const int64_t P = sw ? N : M, Q = sw ? M : N;
    const bool q_rows = (sw ? a_group : b_group) == 1;
    for (const TileCost& t : kTileCosts) {
      if (want ? t.bn != want : (no_pair && t.bn == 256)) continue;
      const int ctas = t.bn == 256 ? 2 : 1;
      const int64_t tiles = (P + 128 * ctas - 1) / (128 * ctas) * ((Q + t.bn - 1) / t.bn);
      for (int c = 1; c <= 8; c *= 2) {
        if (c > 1 && (ctas == 2 || (opts && opts->no_split) || tiles * c > (c > 2 ? have * 7 / 8 : have) ||
                      kt < kMinShare * c))
          break;
        const int64_t workers = have / (ctas * c);
        if (workers < 1) break;
        const int64_t waves = (tiles + workers - 1) / workers, blocks = waves * ((kt + c - 1) / c);
        double ns = blocks * static_cast<double>(q_rows ? t.k_rows : t.k_block);
        const double read = (M + N) * static_cast<double>(K) / kReadGbs;
        if (ns < read) ns = read;
        ns += t.call + (waves - 1) * t.more + (c > 1 ? t.exchange : 0) + (sw ? waves * t.bn * kSwappedNs : 0);
        if (!tile || ns < best) {
          best = ns;
          tile = &t;
          best_c = c;
          swapped = sw != 0;
        }
      }
    }
  }
  if (!tile) return GP_ERR_UNSUPPORTED;   // (width 256 forced on one SM: a pair of CTAs does not fit)
  const int64_t p_rows = swapped ? N : M, q_rows = swapped ? M : N;
  p->dtype = GP_PLAN_FP8;
  p->layout = swapped;
  p->variant = GP_PIPELINED;
  p->threads = kThreads;
  p->persistent = 1;
  p->kernel = tile->bn == 256 ? "fp8_pair_ring" : "fp8_ring";
  switch (tile->bn) {
    case 16: shape_of<16, false>(p); break;
    case 32: shape_of<32, false>(p); break;
    case 64: shape_of<64, false>(p); break;
    case 128: shape_of<128, false>(p); break;
    default: shape_of<256, true>(p); break;
  }
  p->tiles = (p_rows + p->bm - 1) / p->bm * ((q_rows + p->bn - 1) / p->bn);
  p->k_tiles = kt;
  if (p->tiles > kMaxTiles) return GP_ERR_SIZE;
  p->dp_tiles = static_cast<int32_t>(p->tiles);
  p->k_splits = best_c;
  p->raster_gm = 8;
  p->compute_load_ratio = 2.0 * p->bm * p->bn / (p->bm + p->bn);
  const int64_t ctas = p->cta_pair ? 2 : best_c, workers = sms / ctas;
  p->grid = static_cast<int32_t>(ctas * (p->tiles < workers ? p->tiles : workers));
  return GP_OK;
}

cudaError_t launch_fp8_gemm(Fp8GemmArgs& a, const void** kernel) {
  const gp_fp8_matrix& Q = a.plan.layout ? a.A : a.B;
  switch (a.plan.bn) {
    case 16: return launch_ring<16, true, false>(a, kernel);
    case 32: return launch_ring<32, true, false>(a, kernel);
    case 64: return launch_ring<64, true, false>(a, kernel);
    case 128: return Q.group == 1 ? launch_ring<128, true, false>(a, kernel) : launch_ring<128, false, false>(a, kernel);
    default: return Q.group == 1 ? launch_ring<256, true, true>(a, kernel) : launch_ring<256, false, true>(a, kernel);
  }
}

cudaError_t fp8_fit_pairs(gp_plan* plan) {
  if (!plan->cta_pair) return cudaSuccess;
  int pairs = 0;
  const cudaError_t e = pair_capacity(&pairs);
  if (e == cudaSuccess && 2 * pairs < plan->grid) plan->grid = 2 * pairs;
  return e;
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
