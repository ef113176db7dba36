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
//   warps 0, 2, 3   TMA producers, each of every third ring slot (a slot is 64 of the
//              summed axis): one thread issues a slot's loads in about 230 ns, which
//              is longer than the products of a 128 x 128 tile's slot take
//   warp 1     allocates TMEM and issues tcgen05.mma (kind::f16, FP32 in TMEM)
//   warps 4+   write the outputs from one TMEM buffer while the next tile's products
//              run into the other
// PAIR: a cluster of two CTAs shares a 256 x 256 tile (M = 256 instructions).  The
// tiles after the last full round go as two halves of their columns each, where all
// of those make one round: 4096 x 4096 outputs are 256 tiles, 3.37 rounds of 76
// pairs, and take 3.5 instead of 4.
//
// The tensor cores cut their FP32 sums instead of rounding them, always towards
// zero (measured here on operands of one sign: 6e-6 relative after 1024 of K, 5.2e-5
// after 8192, 4.2e-4 after 65536).  Where FP32 leaves, or the scales of 8-bit codes,
// the accumulator is handed over every 768 of K and added to sums in registers; where
// 16 bits leave, before the loss could reach their rounding (ffn_restart).
#pragma once
#include <atomic>
#include <cstring>
#include "ffn_math.cuh"
#include "fp8_rows.cuh"
#include "gp_device.cuh"

namespace gp {

constexpr int kRingLaunchRegs = 96;        // registers per thread at launch, where warps trade them
constexpr int kRingMax = 8;
constexpr int kRingProducers = 3;          // threads that issue loads

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

// How the sums leave.  A lane has 32 columns of its own row at a time in
// registers, and reads and writes the row's memory itself, a whole 32-byte sector
// per access: no shared memory, whose bandwidth the operands take (through it, a
// 256 x 256 tile of BF16 took 8000 cycles to leave, beside 16,400 of products at K
// = 2048).  kStream: straight from TMEM, in a loop.  kHold: a warp takes 64 sums
// per lane to registers, hands the buffer back and works on them: it can add up
// several hand-overs, and sees half of a group of 128 columns.  kCodes: the same
// where 8-bit codes are kept, a kernel of its own as FP32 outputs would pay for its
// registers (4096^3 with both gradients 168 -> 172 us).  kLong: the same where 16 bits
// leave and the summed axis is longer than one accumulator takes.
// L2 takes a request per row and access, beside those of the operands' loads.
// Where more bytes leave than in 16 bits, lanes therefore exchange pieces first and
// write longer runs of each row: FP32 128 bytes by four lanes (4096 x 4096 over
// 4096 added to an addend 106 -> 92 us), what stands beside codes 64 bytes and the
// codes 32 by two (4096 x 8192 x 2056 122 -> 112 us).  It does not pay where 16
// bits leave alone (8192 x 8192 x 4096 271 us either way) nor in a gated product,
// where it costs registers (288 -> 289 us, 323 -> 331 kept up).
enum RingOut { kStream = 0, kHold = 1, kCodes = 2, kLong = 3 };

template <int BN, bool PAIR, RingOut OUT>
struct RingShape {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int A_ROWS = 128;                     // per CTA
  static constexpr int B_ROWS = BN / CTAS;
  static_assert(B_ROWS == 128, "a CTA's share of b is two blocks of 64");
  static constexpr int TILE_ROWS = A_ROWS * CTAS;
  static constexpr int A_BYTES = A_ROWS * kFfnBK * 2;
  static constexpr int STAGE = (A_ROWS + B_ROWS) * kFfnBK * 2;
  static constexpr int EPI_WARPS = OUT != kStream ? BN / 16 : 8;
  static constexpr int EPI_COLS = 4 * BN / EPI_WARPS;    // TMEM columns of each, over 32 rows
  static_assert(OUT == kStream || EPI_COLS == 64, "held sums");
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr int SHARED_MAX = OUT != kStream ? EPI_WARPS * 32 * 8 : 0;   // maxima that warps show each other
  static constexpr int FIXED = SHARED_MAX + kRingBarrierBytes + kSmemAlignSlack;
  static constexpr int FIT = (kSmemPerCtaMax - FIXED) / STAGE;
  static constexpr int STAGES = FIT < kRingMax ? FIT : kRingMax;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static_assert(STAGES > kRingProducers, "a slot for each producer");
  // Sixteen warps that hold 64 sums per thread take registers for them from the other four.
  static constexpr bool SPLIT_REGS = THREADS == 640;
  static constexpr int EPI_REGS = 104, OTHER_REGS = 64;
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
  int32_t whole;             // tiles that are not cut in halves: the first ones
  int32_t items;             // these, and the halves
  uint32_t idesc, idesc_half;
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

// Loads of a box of three dimensions, as tma_load_2d and tma_load_2d_pair.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster_addr, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// How 128 rows of an MN-major operand come: as one box of two planes of 64 (0) where
// its last whole plane reaches that far, or it ends with one; else in boxes of 64,
// of which the second is left out where no row of it exists (its slot then holds
// what it held: those rows' sums are not written).
__device__ __forceinline__ int mn_boxes(int row, int rows) {
  if (rows % 64 == 0 || row + 128 <= (rows & ~63)) return 0;
  return row + 64 >= rows ? 1 : 2;
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

// One of the threads that issue loads: every kRingProducers-th ring slot is its own.
struct RingProducer {
  int which;               // 0 .. kRingProducers - 1, or -1
  int slot;
  uint32_t phase = 0;
  int issued = 0, lost = -1;   // slots so far, and the one whose load the test hook skipped
  __device__ __forceinline__ explicit RingProducer(int warp)
      : which(warp == 0 ? 0 : (warp == 2 || warp == 3 ? warp - 1 : -1)), slot(which) {}
  __device__ __forceinline__ void advance(int stages) {
    ++issued;
    if ((slot += kRingProducers) >= stages) {
      slot -= stages;
      phase ^= 1u;
    }
  }
  // Loads still in flight land in shared memory: wait for them before exit.
  __device__ __forceinline__ void drain(uint64_t* full, int stages, const KernelCtl& ctl) {
    CtaCtl never_abort{0};
    for (int i = max(0, issued - stages / kRingProducers - 1); i < issued; ++i) {
      const int n = which + i * kRingProducers;
      if (i != lost) mbar_wait(full + n % stages, static_cast<uint32_t>((n / stages) & 1), ctl, &never_abort, kSiteDrain);
    }
  }
};

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

// What a worker works on: a tile, or half of its columns.
struct RingItem {
  int problem, rb, cb;
  int half;              // 0 or 1, or -1: the whole tile
};
__device__ __forceinline__ RingItem ring_item(int item, const RingParams& g, int row_blocks, int col_blocks) {
  RingItem t;
  int tile = item;
  t.half = -1;
  if (item >= g.whole) {
    tile = g.whole + ((item - g.whole) >> 1);
    t.half = (item - g.whole) & 1;
  }
  const int per = row_blocks * col_blocks;
  t.problem = tile >= per ? 1 : 0;
  ring_tile(tile - t.problem * per, row_blocks, col_blocks, g.raster, t.rb, t.cb);
  return t;
}

// ---------------------------------------------------------------------------
// sums to outputs: a warp has 32 rows, a lane one of them
// ---------------------------------------------------------------------------
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// The values of a row that 32 bytes hold (16 or 8), in memory's form; `n` of them exist (that many or less), `align` says
// whether rows begin on boundaries of 32 bytes (2), 16 (1) or their own size (0).
template <typename T>
struct Sector {
  static constexpr int N = 32 / static_cast<int>(sizeof(T));
  uint32_t w[8];
};
template <typename T>
__device__ __forceinline__ void load_sector(Sector<T>& r, const T* p, int n, int align) {
  constexpr int PER16 = Sector<T>::N / 2;
  if (n >= Sector<T>::N && align == 2) {
    ld_global_v8(p, r.w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = i * PER16;
    if (align && at + PER16 <= n) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + at);
      memcpy(r.w + 4 * i, &v, 16);
      continue;
    }
    T t[PER16];
#pragma unroll
    for (int k = 0; k < PER16; ++k) {
      from_f32(0.f, t[k]);
      if (at + k < n) t[k] = p[at + k];
    }
    memcpy(r.w + 4 * i, t, 16);
  }
}
template <typename T>
__device__ __forceinline__ float sector_value(const Sector<T>& r, int i) {
  if constexpr (sizeof(T) == 4) return word_lo<T>(r.w[i]);
  return i & 1 ? word_hi<T>(r.w[i / 2]) : word_lo<T>(r.w[i / 2]);
}
template <typename T>
__device__ __forceinline__ void store_sector(T* p, const float* v, int n, int align) {
  constexpr int N = Sector<T>::N, PER16 = N / 2;
  T t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) from_f32(v[i], t[i]);
  uint32_t w[8];
  memcpy(w, t, 32);
  if (n >= N && align == 2) {
    st_global_v8(p, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (align && (i + 1) * PER16 <= n) {
      *reinterpret_cast<uint4*>(p + i * PER16) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      continue;
    }
#pragma unroll
    for (int k = i * PER16; k < (i + 1) * PER16; ++k)
      if (k < n) p[k] = t[k];
  }
}
// 32 neighbouring values.
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float* v, int n, int align) {
#pragma unroll
  for (int i = 0; i < 32; i += Sector<T>::N) store_sector(p + i, v + i, n - i, align);
}

// Sixteen codes of a row, `n` of which exist.
__device__ __forceinline__ void store_codes16(uint8_t* p, const uint32_t* w, int n) {
  if (n >= 16) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
}

// Adds 32 columns' bias, of which a lane fetches one.
template <typename T>
__device__ __forceinline__ void add_bias(float* v, const FfnOut& o, int lane, int64_t first, int64_t cols) {
  const int64_t c = first + lane;
  float b = 0.f;
  if (c < cols) b = o.bias_f32 ? static_cast<const float*>(o.bias)[c] : to_f32(static_cast<const T*>(o.bias)[c]);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, b, i);
}

// LANES neighbouring lanes hold a row each, in LANES pieces of R words.  Pieces change hands: lane b, which held piece k of
// its row in w[R k ..], then has piece b of row k there, so that the lanes reach a longer run of each row together.  Its own
// inverse.
template <int LANES, int R, typename W>
__device__ __forceinline__ void exchange(W* w, int lane) {
#pragma unroll
  for (int step = 1; step < LANES; step *= 2) {
    const bool upper = lane & step;
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
      if (k & step) continue;
      const int lo = R * k, hi = R * (k | step);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const W got = __shfl_xor_sync(0xffffffffu, upper ? w[lo + i] : w[hi + i], step);
        if (upper) w[lo + i] = got; else w[hi + i] = got;
      }
    }
  }
}

// 32 columns from `first` on of a warp's rows, of which this lane holds `row`, added to FP32's addend (if there is one that
// the sums did not begin with) and written in whole lines.  All 32 columns exist, rows begin on 32-byte boundaries.
__device__ __forceinline__ void write_lines(const FfnOut& o, int p, float (&v)[32], int lane, int64_t row, int64_t rows,
                                            int64_t first, bool with_addend) {
  exchange<4, 8>(v, lane);
  const int64_t row0 = row - (lane & 3), col = first + 8 * (lane & 3);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (row0 + k < rows) {
      if (with_addend && o.add[p]) {
        Sector<float> was;
        ld_global_v8(static_cast<const float*>(o.add[p]) + (row0 + k) * o.ld_add[p] + col, was.w);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[8 * k + c] += __uint_as_float(was.w[c]);
      }
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = __float_as_uint(v[8 * k + c]);
      st_global_v8(static_cast<float*>(o.out[p]) + (row0 + k) * o.ld_out[p] + col, w);
    }
  }
}

// The same in 16 bits and without an addend, 64 bytes of a row by two lanes.
template <typename T>
__device__ __forceinline__ void write_half_lines(const FfnOut& o, int p, const float (&v)[32], int lane, int64_t row,
                                                 int64_t rows, int64_t first) {
  T t[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) from_f32(v[i], t[i]);
  uint32_t w[16];
  memcpy(w, t, 64);
  exchange<2, 8>(w, lane);
  const int64_t row0 = row - (lane & 1), col = first + 16 * (lane & 1);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (row0 + k < rows) {
      uint32_t s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = w[8 * k + i];
      st_global_v8(static_cast<T*>(o.out[p]) + (row0 + k) * o.ld_out[p] + col, s);
    }
  }
}

// out = act(v) + addend, and v itself where it is kept: a lane's 32 columns.
template <typename T, typename O>
__device__ __forceinline__ void emit_row(const FfnOut& o, int p, float (&v)[32], int64_t row, int64_t first, int n,
                                         bool with_addend = true) {
  constexpr int N = Sector<O>::N;
  O* const out = static_cast<O*>(o.out[p]) + row * o.ld_out[p] + first;
  if (o.keep[0]) store_row(static_cast<T*>(o.keep[0]) + row * o.ld_keep[0] + first, v, n, o.vec);
  activate_all(v, o.act);
  if (o.add[p] && with_addend) {
    // 16-bit addends all at once, FP32 ones sector by sector, as registers allow; each before its output is written, which
    // may be the same memory
    const O* const add = static_cast<const O*>(o.add[p]) + row * o.ld_add[p] + first;
    constexpr int AT_ONCE = sizeof(O) == 2 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 32; i += AT_ONCE * N) {
      Sector<O> was[AT_ONCE];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) load_sector(was[k], add + i + k * N, n - i - k * N, o.vec);
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
#pragma unroll
        for (int c = 0; c < N; ++c) v[i + k * N + c] += sector_value(was[k], c);
        store_sector(out + i + k * N, v + i + k * N, n - i - k * N, o.vec);
      }
    }
    return;
  }
  store_row(out, v, n, o.vec);
}

// An FP32 addend's 64 columns, where the sums begin.
__device__ __forceinline__ void load_addend(float (&acc)[2][32], const FfnOut& o, int p, int lane, int64_t row, int64_t rows,
                                            int64_t col0, int64_t cols) {
  const float* const add = static_cast<const float*>(o.add[p]);
  if (o.vec == 2 && col0 + 64 <= cols) {
    const int64_t row0 = row - (lane & 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row0 + k < rows) {
          Sector<float> s;
          ld_global_v8(add + (row0 + k) * o.ld_add[p] + col0 + 32 * j + 8 * (lane & 3), s.w);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j][8 * k + i] = __uint_as_float(s.w[i]);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) exchange<4, 8>(acc[j], lane);
    return;
  }
  if (row >= rows) return;
  const int n = cols - col0 < 64 ? static_cast<int>(cols - col0) : 64;   // (may be < 0)
#pragma unroll
  for (int i = 0; i < 64; i += 8) {
    Sector<float> s;
    load_sector(s, add + row * o.ld_add[p] + col0 + i, n - i, o.vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i >> 5][(i & 31) + k] = sector_value(s, k);
  }
}

// h = act(g) * u, and g and u themselves where they are kept: a lane's 32 columns.
template <typename T>
__device__ __forceinline__ void emit_gated(const FfnOut& o, float (&g)[32], const float* u, int64_t row, int64_t first, int n) {
  if (o.keep[0]) {
    store_row(static_cast<T*>(o.keep[0]) + row * o.ld_keep[0] + first, g, n, o.vec);
    store_row(static_cast<T*>(o.keep[1]) + row * o.ld_keep[1] + first, u, n, o.vec);
  }
  activate_all(g, o.act);
#pragma unroll
  for (int i = 0; i < 32; ++i) g[i] *= u[i];
  store_row(static_cast<T*>(o.out[0]) + row * o.ld_out[0] + first, g, n, o.vec);
}

__device__ __forceinline__ int columns_left(int64_t first, int64_t cols) {
  return cols - first < 32 ? static_cast<int>(cols - first) : 32;
}

// 32 columns of TMEM, or zeros.
__device__ __forceinline__ void load_sums(float (&v)[32], uint32_t src, bool sums) {
  uint32_t s[32];
  if (sums) {
    tmem_ld_32x32b_x32(src, s);
    tmem_wait_ld();
    regs_after_wait(s);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = sums ? __uint_as_float(s[i]) : 0.f;
}

// A tile's outputs straight from TMEM: `outs` columns of the warp's rows, 32 at a time.  `src`: the first sum's address (sums
// false: there are none, all are 0); `other`: how far behind it the second weight's lie; release(): called when the last
// has been read.
template <bool GATED, typename T, typename Release>
__device__ __forceinline__ void stream_out(const RingParams& g, int p, int outs, uint32_t src, uint32_t other, bool sums, Release release,
                                           int lane, int64_t row, int64_t col0) {
  const FfnOut& o = g.o;
  const int64_t cols = g.cols;
  if (col0 >= cols) {
    if (sums) release();
    return;
  }
#pragma unroll 1
  for (int j = 0; j < outs / 32; ++j) {
    const int64_t first = col0 + j * 32;
    if (first >= cols) break;
    float v[32], u[GATED ? 32 : 1];
    load_sums(v, src + j * 32, sums);
    if constexpr (GATED) load_sums(u, src + other + j * 32, sums);
    if (sums && (j + 1 == outs / 32 || first + 32 >= cols)) release();
    if (!GATED && o.bias) add_bias<T>(v, o, lane, first, cols);
    if (row < g.rows) {
      if constexpr (GATED)
        emit_gated<T>(o, v, u, row, first, columns_left(first, cols));
      else
        emit_row<T, T>(o, p, v, row, first, columns_left(first, cols));
    }
    __syncwarp();
  }
}

// The larger magnitude, a NaN before any number.
__device__ __forceinline__ float max_abs(float m, float x) {
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmax.NaN.f32 %0, %0, t;\n\t}" : "+f"(m) : "f"(x));
  return m;
}

template <int N>
__device__ __forceinline__ float max_abs_of(const float (&v)[N]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};   // four chains
#pragma unroll
  for (int i = 0; i < N; ++i) m[i & 3] = max_abs(m[i & 3], v[i]);
  return max_abs(max_abs(m[0], m[1]), max_abs(m[2], m[3]));
}

// The largest over the `warps` warps that hold a group of 128 columns together: their slots of shared memory lie 4 warps
// apart, this one's is the `which`-th.  All of them come here for every tile that is kept in 8 bits.
constexpr int kMaxSlot = 32 * 8;
template <int N>
__device__ __forceinline__ void share_max(float (&m)[N], uint32_t slot, int lane, int which, int warps, int barrier) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + (i * 32 + lane) * 4), "f"(m[i]) : "memory");
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
  for (int w = 0; w < warps; ++w) {
    if (w == which) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float x;
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(slot + (w - which) * 4 * kMaxSlot + (i * 32 + lane) * 4) : "memory");
      m[i] = max_abs(m[i], x);
    }
  }
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");   // (read before the next tile's)
}

// 32 values as codes, to a row's columns from `first` on, n of which exist.
__device__ __forceinline__ void emit_codes(const FfnCodes& q, const float* v, float inv, int64_t row, int64_t first, int n) {
  uint8_t* const p = q.data + row * q.ld + first;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* x = v + 16 * i + 4 * k;
      w[k] = fp8x4<false>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
    store_codes16(p + 16 * i, w, n - 16 * i);
  }
}
// The same of a warp's rows, of which this lane holds `row`, where all 32 columns exist: a sector of a row by two lanes.
__device__ __forceinline__ void emit_code_lines(const FfnCodes& q, const float* v, float inv, int lane, int64_t row, int64_t rows,
                                                int64_t first) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = fp8x4<false>(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
  exchange<2, 4>(w, lane);
  const int64_t row0 = row - (lane & 1);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (row0 + k < rows) store_codes16(q.data + (row0 + k) * q.ld + first + 16 * (lane & 1), w + 4 * k, 16);
}

// out = act(s + bias) + addend of a lane's 64 columns; `part`: which 64 of the tile's columns.  write false: nothing is
// written (the row does not exist, or its sums did not come); `whole`: this but for the row; `added`: the sums began with
// the addend.
template <typename T, typename O, bool CODES>
__device__ __forceinline__ void finish_linear(const RingParams& g, int p, float (&acc)[2][32], uint32_t slot, int lane,
                                              int quarter, int part, int64_t row, int64_t col0, bool whole, bool added) {
  const FfnOut& o = g.o;
  const int64_t cols = g.cols;
  const bool write = whole && row < g.rows;
  if (o.bias) {
#pragma unroll
    for (int j = 0; j < 2; ++j) add_bias<T>(acc[j], o, lane, col0 + 32 * j, cols);
  }
  if constexpr (CODES) {
    if (col0 + 64 > cols) {   // (an infinity times a column that is not there is NaN)
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (col0 + i >= cols) acc[i >> 5][i & 31] = 0.f;
    }
    float most[1] = {max_abs(max_abs_of(acc[0]), max_abs_of(acc[1]))};
    share_max(most, slot, lane, part & 1, 2, 2 + quarter * 2 + (part >> 1));
    const GroupScale s = group_scale(__float_as_uint(most[0]), 448.f);
    const FfnCodes& q = o.codes[0];
    if (whole && col0 + 64 <= cols) {
      if (write && (part & 1) == 0) q.scales[row * q.stride_row + (col0 >> 7) * q.stride_col] = s.scale;
#pragma unroll
      for (int j = 0; j < 2; ++j) emit_code_lines(q, acc[j], s.inv, lane, row, g.rows, col0 + 32 * j);
    } else if (write && col0 < cols) {
      if ((part & 1) == 0) q.scales[row * q.stride_row + (col0 >> 7) * q.stride_col] = s.scale;
#pragma unroll
      for (int j = 0; j < 2; ++j) emit_codes(q, acc[j], s.inv, row, col0 + 32 * j, columns_left(col0 + 32 * j, cols));
    }
  }
  if constexpr (sizeof(O) == 4) {
    if (o.vec == 2 && col0 + 64 <= cols) {
      // (warps whose sums did not come, or that have no columns of a half tile, have `whole` false in all lanes)
      if (!whole) return;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!CODES && o.keep[0] && write)
          store_row(static_cast<T*>(o.keep[0]) + row * o.ld_keep[0] + col0 + 32 * j, acc[j], 32, o.vec);
        activate_all(acc[j], o.act);
        write_lines(o, p, acc[j], lane, row, g.rows, col0 + 32 * j, !added);
      }
      return;
    }
  }
  if constexpr (sizeof(O) == 2 && CODES) {
    if (o.vec == 2 && col0 + 64 <= cols && !o.add[p]) {   // (beside codes nothing else is kept)
      if (!whole) return;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        activate_all(acc[j], o.act);
        write_half_lines<O>(o, p, acc[j], lane, row, g.rows, col0 + 32 * j);
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (write && col0 + 32 * j < cols)
      emit_row<T, O>(o, p, acc[j], row, col0 + 32 * j, columns_left(col0 + 32 * j, cols), !added);
  __syncwarp();
}

// h = act(g) * u of a lane's 32 columns: acc[0] are g's sums, acc[1] u's.  `part`: which 32 of the tile's columns, four of
// which are a group of 128.
template <typename T, bool CODES>
__device__ __forceinline__ void finish_gated(const RingParams& g, float (&acc)[2][32], uint32_t slot, int lane, int quarter,
                                             int part, int64_t row, int64_t col0, bool write) {
  const FfnOut& o = g.o;
  const int64_t cols = g.cols;
  if constexpr (CODES) {
    if (col0 + 32 > cols) {   // (an infinity times a column that is not there is NaN)
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i >= cols) acc[0][i] = acc[1][i] = 0.f;
    }
    float most[2] = {max_abs_of(acc[0]), max_abs_of(acc[1])};
    share_max(most, slot, lane, part, 4, 2 + quarter);
    if (write && col0 < cols) {
      const int n = columns_left(col0, cols);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const GroupScale s = group_scale(__float_as_uint(most[j]), 448.f);
        const FfnCodes& q = o.codes[j];
        if (part == 0) q.scales[row * q.stride_row + (col0 >> 7) * q.stride_col] = s.scale;
        emit_codes(q, acc[j], s.inv, row, col0, n);
      }
    }
  }
  if (write && col0 < cols) emit_gated<T>(o, acc[0], acc[1], row, col0, columns_left(col0, cols));
  __syncwarp();
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
// Maps: a of the first and second source or product, b likewise, or of the two weights of a gated product.
struct RingMaps {
  CUtensorMap a[2], b[2];
  CUtensorMap a64[2], b64[2];          // in boxes of 64 of their rows: an MN-major operand's end, half tiles
};

template <int BN, bool PAIR, RingOut OUT, bool GATED, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(RingShape<BN, PAIR, OUT>::THREADS, 1)
    ffn_ring_kernel(const __grid_constant__ RingMaps maps, const __grid_constant__ RingParams g) {
  using Sh = RingShape<BN, PAIR, OUT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* maxima = ring + Sh::STAGES * Sh::STAGE;
  RingBarriers* bar = reinterpret_cast<RingBarriers*>(maxima + Sh::SHARED_MAX);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // (uniform for the compiler too)
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int worker = static_cast<int>(blockIdx.x) / Sh::CTAS;
  const int workers = static_cast<int>(gridDim.x) / Sh::CTAS;
  constexpr int TILE_COLS = GATED ? BN / 2 : BN;
  const int row_blocks = (g.rows + Sh::TILE_ROWS - 1) / Sh::TILE_ROWS;
  const int col_blocks = (g.cols + TILE_COLS - 1) / TILE_COLS;
  const int items = g.items;
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
  RingProducer prod(warp);

  if (warp < 4) {
    if (Sh::SPLIT_REGS) regs_decrease<Sh::OTHER_REGS>();
    if (warp != 1 && lane == 0) {
      // ---------------- producers (every CTA) ----------------
      const int lose_item = g.ctl.inject_lost_load ? items - 1 : -1;   // test hook: this tile's last load never comes
      bool ok = true;
      int kb = prod.which;
      for (int item = worker; ok && item < items; item += workers, kb -= kt) {
        const RingItem t = ring_item(item, g, row_blocks, col_blocks);
        const int a_row = t.rb * Sh::TILE_ROWS + static_cast<int>(rank) * Sh::A_ROWS;
        const bool half = PAIR && t.half >= 0;
        const int b_row = !half ? (GATED ? t.cb * TILE_COLS : t.cb * BN + static_cast<int>(rank) * Sh::B_ROWS)
                                : t.cb * TILE_COLS + t.half * (TILE_COLS / 2) + (GATED ? 0 : static_cast<int>(rank) * 64);
        // boxes of either operand, and the bytes of a slot over all CTAs
        const int a_boxes = A_MN ? mn_boxes(a_row, g.rows) : 0, b_boxes = B_MN && !half ? mn_boxes(b_row, g.cols) : 0;
        uint32_t bytes = Sh::CTAS * (half ? Sh::STAGE - 8192 : Sh::STAGE);
        if (A_MN) {
#pragma unroll
          for (int r = 0; r < Sh::CTAS; ++r)
            if (mn_boxes(t.rb * Sh::TILE_ROWS + r * Sh::A_ROWS, g.rows) == 1) bytes -= 8192;
        }
        if (B_MN && !half) {
#pragma unroll
          for (int r = 0; r < Sh::CTAS; ++r)
            if (mn_boxes(t.cb * BN + r * Sh::B_ROWS, g.cols) == 1) bytes -= 8192;
        }
        for (; kb < kt; kb += kRingProducers) {
          const int s = prod.slot;
          if (!mbar_wait(&bar->empty[s], prod.phase ^ 1u, g.ctl, cta, kSiteProducerEmpty) || cta->abort) { ok = false; break; }
          const int second = kb >= g.kt ? 1 : 0;      // the second source
          const int k = (kb - second * g.kt) * kFfnBK;
          const CUtensorMap* ma = &maps.a[t.problem | second];
          const int which_b = GATED ? static_cast<int>(rank) : second;   // (two products share b)
          const CUtensorMap* mb = &maps.b[which_b];
          const uint32_t a_at = smem_u32(ring + s * Sh::STAGE), b_at = a_at + Sh::A_BYTES;
          const uint32_t full = PAIR ? mapa_shared(smem_u32(&bar->full[s]), 0) : 0u;
          auto load = [&](uint32_t at, const CUtensorMap* m, int x, int y) {
            if (PAIR)
              tma_load_2d_pair(at, m, full, x, y);
            else
              tma_load_2d(at, m, &bar->full[s], x, y);
          };
          // Two boxes of 8 KB where one of 16 KB would do cost time in the TMA unit: 4096 x 8192 x 4096 142 us with two
          // boxes per slot, 161 with four.
          auto load_mn = [&](uint32_t at, const CUtensorMap* planes, const CUtensorMap* m, int boxes, int row) {
            if (boxes) {
              load(at, m, row, k);
              if (boxes == 2) load(at + 8192, m, row + 64, k);
            } else if (PAIR) {
              tma_load_3d_pair(at, planes, full, 0, k, row >> 6);
            } else {
              tma_load_3d(at, planes, &bar->full[s], 0, k, row >> 6);
            }
          };
          if (item == lose_item && kb == kt - 1) {
            prod.lost = prod.issued;
          } else {
            // (the even CTA's barrier counts the bytes of both CTAs' loads)
            if (rank == 0) mbar_arrive_expect_tx(&bar->full[s], bytes);
            if (A_MN)
              load_mn(a_at, ma, &maps.a64[t.problem | second], a_boxes, a_row);
            else
              load(a_at, ma, k, a_row);
            if (half) {
              load(b_at, &maps.b64[which_b], B_MN ? b_row : k, B_MN ? k : b_row);
            } else if (B_MN) {
              load_mn(b_at, mb, &maps.b64[which_b], b_boxes, b_row);
            } else if (GATED && !PAIR) {
              load(b_at, mb, k, b_row);
              load(b_at + 8192, &maps.b[1], k, b_row);
            } else {
              load(b_at, mb, k, b_row);
            }
          }
          prod.advance(Sh::STAGES);
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (the even CTA of a pair) ----------------
      // One lane walks the loop (with the warp's votes on each wait a 128 x 64
      // tile's slot took 265 ns instead of 200).
      int s = 0, a = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      if (ring_elect_one()) {
        const uint32_t ring0 = smem_u32(ring);
        const uint64_t a0 = A_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0);
        const uint64_t b0 = (B_MN ? umma_desc_mn(ring0) : umma_desc_sw128(ring0)) + Sh::A_BYTES / 16;
        // 16 along K: 32 bytes of a K-major row, 16 rows of 128 bytes of an MN-major tile
        constexpr uint32_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;
        for (int item = worker; ok && item < items; item += workers) {
          const uint32_t idesc = item < g.whole ? g.idesc : g.idesc_half;
          for (int kc = 0; ok && kc < kt; kc += g.restart) {
            const int end = min(kc + g.restart, kt);
            if (!mbar_wait(&bar->acc_empty[a], aph ^ 1u, g.ctl, cta, kSiteMmaAccEmpty)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d = tmem + a * BN;
            for (int kb = kc; kb < end; ++kb) {
              // (nothing is issued of a slot that never came)
              if (!mbar_wait(&bar->full[s], ph, g.ctl, cta, kSiteConsumerFull)) { ok = false; break; }
              tc_fence_after();
              const uint64_t da = a0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
              const uint64_t db = b0 + static_cast<uint32_t>(s * Sh::STAGE) / 16;
#pragma unroll
              for (int kk = 0; kk < kFfnBK / 16; ++kk) {
                const uint32_t more = kb > kc || kk > 0;
                if (PAIR)
                  umma_f16_pair(d, da + A_STEP * kk, db + B_STEP * kk, idesc, more);
                else
                  umma_f16(d, da + A_STEP * kk, db + B_STEP * kk, idesc, more);
              }
              if (PAIR) umma_commit_pair(&bar->empty[s], 0x3); else umma_commit(&bar->empty[s]);
              if (++s == Sh::STAGES) { s = 0; ph ^= 1u; }
            }
            if (!ok) break;
            if (PAIR) umma_commit_pair(&bar->acc_full[a], 0x3); else umma_commit(&bar->acc_full[a]);
            if (++a == 2) { a = 0; aph ^= 1u; }
          }
        }
        // fires when every MMA issued above has completed
        if (PAIR) umma_commit_pair(&bar->drain, 0x1); else umma_commit(&bar->drain);
        CtaCtl never_abort{0};
        mbar_wait(&bar->drain, 0, g.ctl, &never_abort, kSiteDrain);
      }
    }
    __syncwarp();
  } else {
    // ---------------- outputs ----------------
    if (Sh::SPLIT_REGS) regs_increase<Sh::EPI_REGS>();
    const int e = warp - 4;
    const int quarter = warp & 3;          // TMEM lanes this warp may access
    const int part = e >> 2;               // which of the tile's columns
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    // its output columns, and the TMEM columns of their sums: a gated product's second weight has its own half of a tile
    // further on.  Of a half tile the streaming warps take half of their columns each, the holding ones all or none.
    constexpr int OUTS = GATED ? Sh::EPI_COLS / 2 : Sh::EPI_COLS;
    int a = 0;
    uint32_t aph = 0;
    bool ok = true;   // after a wait that gave up: nothing is written any more
    const bool add_first = OUT == kHold && !GATED && g.o.out_f32 && g.o.add[0] && g.o.act == GP_ACT_NONE && !g.o.keep[0];
    for (int item = worker; item < items; item += workers) {
      const RingItem t = ring_item(item, g, row_blocks, col_blocks);
      const int problem = t.problem;
      const bool cut = PAIR && t.half >= 0;
      const int outs = cut && OUT == kStream ? OUTS / 2 : OUTS;
      const bool idle = cut && part * outs >= TILE_COLS / 2;
      const uint32_t lo = part * outs, other = cut ? BN / 4 : BN / 2;
      const int64_t row = static_cast<int64_t>(t.rb) * Sh::TILE_ROWS + rank * Sh::A_ROWS + quarter * 32 + lane;
      const int64_t col0 = static_cast<int64_t>(t.cb) * TILE_COLS + (cut ? t.half * (TILE_COLS / 2) : 0) + part * outs;
      if (!GATED && g.o.add[problem] && row < g.rows && !idle && !add_first) {
        // this thread's row of the addend comes into L2 while the products run
        const int size = g.o.out_f32 ? 4 : 2;
        const uint8_t* at = static_cast<const uint8_t*>(g.o.add[problem]) + (row * g.o.ld_add[problem] + col0) * size;
#pragma unroll 1
        for (int i = 0; i < outs && col0 + i < g.cols; i += 128 / size) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i * size));
      }
      auto hand_back = [&]() {
        // the buffer has been read: back to the MMA issuer
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            ring_arrive_cluster_relaxed(mapa_shared(smem_u32(&bar->acc_empty[a]), 0));
          else
            mbar_arrive(&bar->acc_empty[a]);
        }
      };
      if constexpr (OUT == kStream) {
        const bool sums = kt > 0;
        if (sums) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bar->acc_full[a], aph, g.ctl, cta, kSiteEpilogueAccFull));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t src = tmem + lanes + a * BN + lo;
        if (g.o.bf16)
          stream_out<GATED, __nv_bfloat16>(g, problem, outs, src, other, sums, hand_back, lane, row, col0);
        else
          stream_out<GATED, __half>(g, problem, outs, src, other, sums, hand_back, lane, row, col0);
        if (sums && ++a == 2) { a = 0; aph ^= 1u; }
      } else {
        float acc[2][32];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i >> 5][i & 31] = 0.f;
        if constexpr (!GATED) {
          // an FP32 addend with nothing between it and the sums is what they are added to: it comes while the products run
          if (add_first && !idle) load_addend(acc, g.o, problem, lane, row, g.rows, col0, g.cols);
        }
#pragma unroll 1
        for (int kc = 0; kc < kt; kc += g.restart) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bar->acc_full[a], aph, g.ctl, cta, kSiteEpilogueAccFull));
          if (!ok) break;
          tc_fence_after();
          const uint32_t src = tmem + lanes + a * BN + lo;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (idle) break;
            uint32_t v[16];
            tmem_ld_32x32b_x16(src + (j >> 1) * (GATED ? other : 32u) + (j & 1) * 16, v);
            tmem_wait_ld();
            regs_after_wait(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j >> 1][(j & 1) * 16 + i] += __uint_as_float(v[i]);
          }
          hand_back();
          if (++a == 2) { a = 0; aph ^= 1u; }
        }
        const bool whole = ok && !idle, write = whole && row < g.rows;
        const uint32_t slot = smem_u32(maxima) + e * kMaxSlot;
        if constexpr (GATED) {
          if (g.o.bf16)
            finish_gated<__nv_bfloat16, OUT == kCodes>(g, acc, slot, lane, quarter, part, row, col0, write);
          else
            finish_gated<__half, OUT == kCodes>(g, acc, slot, lane, quarter, part, row, col0, write);
        } else {
          const bool f32 = OUT == kHold || (OUT == kCodes && g.o.out_f32);
          if (g.o.bf16) {
            if (f32)
              finish_linear<__nv_bfloat16, float, OUT == kCodes>(g, problem, acc, slot, lane, quarter, part, row, col0, whole, add_first);
            else
              finish_linear<__nv_bfloat16, __nv_bfloat16, OUT == kCodes>(g, problem, acc, slot, lane, quarter, part, row, col0, whole, false);
          } else {
            if (f32)
              finish_linear<__half, float, OUT == kCodes>(g, problem, acc, slot, lane, quarter, part, row, col0, whole, add_first);
            else
              finish_linear<__half, __half, OUT == kCodes>(g, problem, acc, slot, lane, quarter, part, row, col0, whole, false);
          }
        }
      }
    }
  }

  __syncthreads();
  if (cta->abort && prod.which >= 0 && lane == 0) {
    if (PAIR) {
      // this CTA's loads count on the even CTA's barrier: give any still in
      // flight time to land before the pair tears down
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
    } else {
      prod.drain(bar->full, Sh::STAGES, g.ctl);
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

// Map of an operand of `rows` x `summed`, whose boxes hold box_rows of its rows; stored summed axis first where `mn`, in
// boxes of two planes of 64 of its rows, as far as they go whole (no plane: the map is not used).
inline cudaError_t ffn_map(CUtensorMap* m, const FfnProduct& p, const void* base, int64_t ld, int64_t rows, bool mn,
                           int box_rows) {
  const uint64_t row_bytes = static_cast<uint64_t>(ld) * 2;
  if (!mn)
    return make_tmap_2d(m, base, ffn_map_type(p.out), p.summed, rows, row_bytes, kFfnBK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rows < 64) return cudaSuccess;
  return make_tmap_3d(m, base, ffn_map_type(p.out), 64, p.summed, row_bytes, rows / 64, 128, 64, kFfnBK, 2,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same in boxes of 64 of its rows.
inline cudaError_t ffn_map64(CUtensorMap* m, const FfnProduct& p, const void* base, int64_t ld, int64_t rows, bool mn) {
  const uint64_t row_bytes = static_cast<uint64_t>(ld) * 2;
  return mn ? make_tmap_2d(m, base, ffn_map_type(p.out), rows, p.summed, row_bytes, 64, kFfnBK, CU_TENSOR_MAP_SWIZZLE_128B)
            : make_tmap_2d(m, base, ffn_map_type(p.out), p.summed, rows, row_bytes, kFfnBK, 64, CU_TENSOR_MAP_SWIZZLE_128B);
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

template <int BN, bool PAIR, RingOut OUT, bool GATED, bool A_MN, bool B_MN>
cudaError_t launch_ring(FfnProduct& p, const void** kernel) {
  using Sh = RingShape<BN, PAIR, OUT>;
  auto k = ffn_ring_kernel<BN, PAIR, OUT, GATED, A_MN, B_MN>;
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
    for (int i = 0; A_MN && p.rows % 64 != 0 && i < (both ? 2 : 1); ++i)
      if ((e = ffn_map64(&maps.a64[i], p, p.a[i], p.lda[i], p.rows, A_MN)) != cudaSuccess) return e;
    const bool b64 = (PAIR && p.plan.half_tiles) || (B_MN && p.cols % 64 != 0);
    for (int i = 0; b64 && i < (sum || GATED ? 2 : 1); ++i)
      if ((e = ffn_map64(&maps.b64[i], p, p.b[i], p.ldb[i], p.cols, B_MN)) != cudaSuccess) return e;
  }
  RingParams g = {};
  g.o = p.out;
  g.rows = static_cast<int32_t>(p.rows);
  g.cols = static_cast<int32_t>(p.cols);
  g.kt = static_cast<int32_t>((p.summed + kFfnBK - 1) / kFfnBK);
  g.sources = sum ? 2 : 1;
  g.problems = both ? 2 : 1;
  g.restart = ffn_restart(p.out.out_f32 || p.out.codes[0].data, p.out.bf16 != 0);
  g.raster = p.plan.raster_gm;
  g.idesc = umma_idesc_f16(p.out.bf16 != 0, Sh::TILE_ROWS, BN) | (A_MN ? kIdescAMn : 0u) | (B_MN ? kIdescBMn : 0u);
  g.idesc_half = umma_idesc_f16(p.out.bf16 != 0, Sh::TILE_ROWS, BN / 2) | (A_MN ? kIdescAMn : 0u) | (B_MN ? kIdescBMn : 0u);
  g.whole = static_cast<int32_t>(p.plan.tiles) - p.plan.half_tiles;
  g.items = g.whole + 2 * p.plan.half_tiles;
  g.ctl = p.ctl;
  if (Sh::SPLIT_REGS) {
    static std::atomic<int> regs{-1};
    if ((e = check_launch_regs(regs, *kernel)) != cudaSuccess) return e;
  }
  if ((e = ensure_smem_attr(*kernel, Sh::SMEM)) != cudaSuccess) return e;
  RingConfig c(p.plan.grid, Sh::THREADS, Sh::CTAS, Sh::SMEM, p.stream);
  return cudaLaunchKernelEx(&c.cfg, k, maps, g);
}

// The tile of the plan; sums are held where FP32 or 8-bit codes leave, or one accumulator does not take them all.
template <bool GATED, bool A_MN, bool B_MN>
cudaError_t launch_tile(FfnProduct& p, const void** kernel) {
  const bool wide = p.out.out_f32 || p.out.codes[0].data;
  const bool lasting = !wide && p.plan.k_tiles > ffn_restart(false, p.out.bf16 != 0);
  if constexpr (GATED) {   // (8 bits on pairs alone)
    if (wide) return launch_ring<256, true, kCodes, true, A_MN, B_MN>(p, kernel);
    if (lasting)
      return p.plan.cta_pair ? launch_ring<256, true, kLong, true, A_MN, B_MN>(p, kernel)
                             : launch_ring<128, false, kLong, true, A_MN, B_MN>(p, kernel);
    return p.plan.cta_pair ? launch_ring<256, true, kStream, true, A_MN, B_MN>(p, kernel)
                           : launch_ring<128, false, kStream, true, A_MN, B_MN>(p, kernel);
  } else {
    const bool pair = p.plan.cta_pair;
    if constexpr (!A_MN && !B_MN) {   // (values are kept by the forward product)
      if (p.out.codes[0].data)
        return pair ? launch_ring<256, true, kCodes, false, A_MN, B_MN>(p, kernel)
                    : launch_ring<128, false, kCodes, false, A_MN, B_MN>(p, kernel);
    }
    if (wide)
      return pair ? launch_ring<256, true, kHold, false, A_MN, B_MN>(p, kernel)
                  : launch_ring<128, false, kHold, false, A_MN, B_MN>(p, kernel);
    if (lasting)
      return pair ? launch_ring<256, true, kLong, false, A_MN, B_MN>(p, kernel)
                  : launch_ring<128, false, kLong, false, A_MN, B_MN>(p, kernel);
    return pair ? launch_ring<256, true, kStream, false, A_MN, B_MN>(p, kernel)
                : launch_ring<128, false, kStream, false, A_MN, B_MN>(p, kernel);
  }
}

}  // namespace gp
