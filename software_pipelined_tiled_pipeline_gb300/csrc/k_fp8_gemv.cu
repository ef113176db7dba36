// k_fp8_gemv.cu -- gemm_fp8 for a few rows on one side (single-token decoding):
// out[t][n] = sum over K blocks b of sW[n][b] * sX[t][b] * (sum over the block of w[n][k] * x[t][k])
//
// With T rows of x (1, 2 or 4) the weights' bytes are all there is to move, and
// at these sizes the call's length is mostly the way to memory and back.  So no
// tile, no ring and no split: one warp per row of w, each lane 16 bytes of it
// at a time, kAhead of them under way before the first is used, and one
// exchange of sums at the end.  A lane's 16 values lie in one K block, so its
// FP32 sum is scaled once per 16 bytes.  x, already in FP16 pairs (an 8-bit
// value is exact in FP16), comes from shared memory; products are exact in
// FP32 and summed there.
#include <cstring>
#include "fp8_internal.h"
#include "gp_device.cuh"

namespace gp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kAhead = 8;                // 16-byte loads of w under way per lane
constexpr int kStep = 32 * 16;           // values of a row that a warp takes at a time
constexpr int kSlab = 16384;             // values of x held in shared memory at a time, over all of its rows

struct GemvArgs {
  const uint8_t *w, *x;
  const float *sw, *sx;
  int64_t ldw, ldx;
  int64_t sw_row, sw_col, sx_row, sx_col;
  void* c;
  const void* addend;
  int64_t c_row, c_col, add_row, add_col;   // strides of (row of x, row of w)
  int32_t rows, n, K;                       // rows of x, rows of w
  int32_t w_shift, x_shift;                 // log2 of the rows that share a scale
  int32_t w_e5m2, x_e5m2, out_type;
};

template <bool E5M2>
__device__ __forceinline__ uint32_t half2_of(uint32_t pair) {   // two codes (low 16 bits) as two FP16
  uint32_t r;
  const uint16_t p = static_cast<uint16_t>(pair);
  if (E5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(p));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(p));
  return r;
}
__device__ __forceinline__ float2 float2_of(uint32_t h2) {
  __half2 h;
  memcpy(&h, &h2, 4);
  return __half22float2(h);
}

// 16 codes at p, of which the first `valid` lie inside the row; the others become zeros.
__device__ __forceinline__ uint4 load16(const uint8_t* p, int valid) {
  uint4 v;
  if (valid >= 16) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (i < valid) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int T, bool WE5>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const __grid_constant__ GemvArgs a) {
  constexpr int COLS = kSlab / T;                              // values of each row of x per slab
  constexpr int STEPS = COLS / kStep;
  __shared__ __align__(16) uint32_t xs[T * COLS / 2];          // FP16 pairs, 32 KB
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const bool live = n < a.n;
  const uint8_t* wr = a.w + (live ? n : 0) * a.ldw;
  const float* swr = a.sw + ((live ? n : 0) >> a.w_shift) * a.sw_row;
  pdl_launch_dependents();
  // While the work before this kernel finishes, the first weights come into L2
  // (a prefetch writes nothing, and L2 stays coherent with what is still written).
  if (live && lane % 8 == 0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = (i * 32 + lane) * 16;
      if (k < a.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(wr + k));
    }
  }
  pdl_wait();

  float total[T];
#pragma unroll
  for (int t = 0; t < T; ++t) total[t] = 0.f;
  for (int base = 0; base < a.K; base += COLS) {
    const int end = min(base + COLS, a.K);
    const int chunks = (end - base + 15) / 16;                 // 16-byte pieces of a row
    // the first weights are asked for before x is staged
    uint4 v[kAhead];
    float s[kAhead];
    auto fetch = [&](int slot, int step) {
      const int ch = step * 32 + lane;
      v[slot] = make_uint4(0, 0, 0, 0);
      s[slot] = 0.f;
      if (live && ch < chunks) {
        const int k = base + ch * 16;
        v[slot] = load16(wr + k, end - k);
        s[slot] = swr[(k >> 7) * a.sw_col];
      }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < STEPS) fetch(i, i);
    if (base > 0) __syncthreads();                             // the slab before has been read
    for (int i = threadIdx.x; i < T * chunks; i += kThreads) {
      const int t = i / chunks, ch = i - t * chunks;
      const int k = base + ch * 16;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (t < a.rows) q = load16(a.x + t * a.ldx + k, end - k);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.x_e5m2) {
          h[2 * j] = half2_of<true>(w[j]);
          h[2 * j + 1] = half2_of<true>(w[j] >> 16);
        } else {
          h[2 * j] = half2_of<false>(w[j]);
          h[2 * j + 1] = half2_of<false>(w[j] >> 16);
        }
      }
      // piece ch as two halves of 16 bytes, COLS / 16 pieces apart, so that a warp's reads touch all banks
      uint4* dst = reinterpret_cast<uint4*>(xs + t * (COLS / 2));
      dst[ch] = make_uint4(h[0], h[1], h[2], h[3]);
      dst[COLS / 16 + ch] = make_uint4(h[4], h[5], h[6], h[7]);
    }
    __syncthreads();
    const int steps = (chunks + 31) / 32;
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int step = s0 + i;
        if (step >= steps) break;
        const int ch = step * 32 + lane;
        const int k = base + ch * 16;
        const uint4 q = v[i];
        const float sw = s[i];
        if (step + kAhead < steps) fetch(i, step + kAhead);
        if (ch >= chunks) continue;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float f[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = float2_of(half2_of<WE5>(w[j])), hi = float2_of(half2_of<WE5>(w[j] >> 16));
          f[4 * j] = lo.x;
          f[4 * j + 1] = lo.y;
          f[4 * j + 2] = hi.x;
          f[4 * j + 3] = hi.y;
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if (t >= a.rows) break;
          const uint4* src = reinterpret_cast<const uint4*>(xs + t * (COLS / 2));
          const uint4 x0 = src[ch], x1 = src[COLS / 16 + ch];
          const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          float d = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 xf = float2_of(xw[j]);
            d = fmaf(f[2 * j], xf.x, d);
            d = fmaf(f[2 * j + 1], xf.y, d);
          }
          const float sx = a.sx[(t >> a.x_shift) * a.sx_row + (k >> 7) * a.sx_col];
          total[t] = fmaf(d, sx * sw, total[t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) total[t] += __shfl_xor_sync(0xffffffffu, total[t], d);
  }
  if (!live) return;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    if (lane != t || t >= a.rows) continue;
    const int64_t at = t * a.c_row + n * a.c_col, from = t * a.add_row + n * a.add_col;
    float v = total[t];
    if (a.out_type == GP_REAL_BF16) {
      if (a.addend) v += __bfloat162float(static_cast<const __nv_bfloat16*>(a.addend)[from]);
      static_cast<__nv_bfloat16*>(a.c)[at] = __float2bfloat16_rn(v);
    } else if (a.out_type == GP_REAL_F16) {
      if (a.addend) v += __half2float(static_cast<const __half*>(a.addend)[from]);
      static_cast<__half*>(a.c)[at] = __float2half_rn(v);
    } else {
      if (a.addend) v += static_cast<const float*>(a.addend)[from];
      static_cast<float*>(a.c)[at] = v;
    }
  }
}

template <int T>
cudaError_t launch_rows(const GemvArgs& a, cudaStream_t stream, const void** kernel) {
  auto k = a.w_e5m2 ? gemv_kernel<T, true> : gemv_kernel<T, false>;
  *kernel = reinterpret_cast<const void*>(k);
  return launch_dependent(k, dim3(static_cast<unsigned>((a.n + kWarps - 1) / kWarps)), dim3(kThreads), 0, stream, a);
}

}  // namespace

void fp8_gemv_plan(int64_t n, gp_plan* p) {
  p->kernel = "fp8_gemv";
  p->persistent = 0;
  p->bm = kWarps;
  p->bn = kFp8GemvRows;
  p->bk = kStep;
  p->threads = kThreads;
  p->smem_bytes = 0;
  p->tiles = (n + kWarps - 1) / kWarps;
  p->grid = static_cast<int32_t>(p->tiles);
}

cudaError_t launch_fp8_gemv(Fp8GemmArgs& g, const void** kernel) {
  const bool swapped = g.plan.layout != 0;   // the weights are B
  const gp_fp8_matrix& W = swapped ? g.B : g.A;
  const gp_fp8_matrix& X = swapped ? g.A : g.B;
  GemvArgs a = {};
  a.w = static_cast<const uint8_t*>(W.data);
  a.x = static_cast<const uint8_t*>(X.data);
  a.sw = W.scales;
  a.sx = X.scales;
  a.ldw = W.ld;
  a.ldx = X.ld;
  a.sw_row = W.stride_row;
  a.sw_col = W.stride_col;
  a.sx_row = X.stride_row;
  a.sx_col = X.stride_col;
  a.c = g.C;
  a.addend = g.addend;
  a.c_row = swapped ? g.ldc : 1;
  a.c_col = swapped ? 1 : g.ldc;
  a.add_row = swapped ? g.ld_add : 1;
  a.add_col = swapped ? 1 : g.ld_add;
  a.rows = swapped ? g.M : g.N;
  a.n = swapped ? g.N : g.M;
  a.K = g.K;
  a.w_shift = W.group == kFp8Group ? 7 : 0;
  a.x_shift = X.group == kFp8Group ? 7 : 0;
  a.w_e5m2 = W.format == GP_E5M2;
  a.x_e5m2 = X.format == GP_E5M2;
  a.out_type = g.out_type;
  if (a.rows == 1) return launch_rows<1>(a, g.stream, kernel);
  if (a.rows == 2) return launch_rows<2>(a, g.stream, kernel);
  return launch_rows<4>(a, g.stream, kernel);
}

}  // namespace gp
