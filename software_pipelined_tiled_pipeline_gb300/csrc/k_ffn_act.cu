// k_ffn_act.cu -- the element-by-element part of the backward pass, and rows
// laid out for the tensor cores.
//
//   linear: dz = dy * act'(z), dbias = column sums of dz before its rounding
//   gated:  dg = dh * u * act'(g), du = dh * act(g), h = act(g) * u
//
// z, g and u come in 16 bits or as 8-bit codes with a scale for each row's 128
// values.  A block takes a strip of 256 columns and a part of the rows, a warp
// every eighth of these, a lane eight columns; the bias gradient is summed in
// FP32 per lane, over the block's warps and, by a second kernel, over the parts,
// each in a fixed order.  HBM bounds it: two bytes in and out per value, one
// for each 8-bit one.
#include <algorithm>
#include "ffn_math.cuh"
#include "fp8_rows.cuh"

namespace gp {
namespace {

constexpr int kActThreads = 256, kActWarps = 8, kActStrip = 256;

// Two 8-bit codes (the lower first) as FP32.
__device__ __forceinline__ float2 decode2(uint32_t codes, bool e5m2) {
  uint32_t h;
  const uint16_t c = static_cast<uint16_t>(codes);
  if (e5m2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  __half2 v;
  memcpy(&v, &h, 4);
  return __half22float2(v);
}

// Eight kept values of a row, as they lie in memory and (below) as FP32.
template <typename T, bool FP8>
struct Kept {
  Raw8<T> r;
};
template <typename T>
struct Kept<T, true> {
  uint2 c;
  float scale;
};

template <typename T, bool FP8>
__device__ __forceinline__ void load_kept(Kept<T, FP8>& k, const void* z, int64_t ldz, const FfnCodes& q, int64_t row, int c,
                                          int cols, bool vec) {
  if constexpr (FP8) {
    const uint8_t* p = q.data + row * q.ld;
    // (with rows off 16-byte boundaries a lane past the end still holds columns of its group)
    k.scale = (c & ~127) < cols ? q.scales[row * q.stride_row + (c >> 7) * q.stride_col] : 0.f;
    if (vec && c + 8 <= cols) {
      k.c = *reinterpret_cast<const uint2*>(p + c);
    } else {
      const Eight e = eight_columns(c, vec);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e.first + i * e.stride < cols) w[i >> 2] |= static_cast<uint32_t>(p[e.first + i * e.stride]) << (8 * (i & 3));
      k.c = make_uint2(w[0], w[1]);
    }
  } else {
    load8(k.r, static_cast<const T*>(z) + row * ldz, c, cols, vec);
  }
}
template <typename T, bool FP8>
__device__ __forceinline__ void widen_kept(float (&v)[8], const Kept<T, FP8>& k, bool e5m2) {
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = decode2((i < 2 ? k.c.x : k.c.y) >> (16 * (i & 1)), e5m2);
      v[2 * i] = f.x * k.scale;
      v[2 * i + 1] = f.y * k.scale;
    }
  } else {
    unpack8(k.r, v);
  }
}

__device__ __forceinline__ void slopes(float (&z)[8], float (&d)[8], int act) {
  switch (act) {
#define GP_SLOPE_LOOP(A)                          \
  case A:                                         \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) { \
      const ActSlope s = activate_slope(z[i], A); \
      z[i] = s.a;                                 \
      d[i] = s.d;                                 \
    }                                             \
    break;
    GP_SLOPE_LOOP(GP_ACT_RELU)
    GP_SLOPE_LOOP(GP_ACT_GELU)
    GP_SLOPE_LOOP(GP_ACT_GELU_TANH)
    GP_SLOPE_LOOP(GP_ACT_SILU)
    GP_SLOPE_LOOP(GP_ACT_SIGMOID)
    default:
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = 1.f;
#undef GP_SLOPE_LOOP
  }
}

// The rows of part `part` of `parts`: whole multiples of the warps each.
struct Rows {
  int64_t from, to;
};
__device__ __forceinline__ Rows rows_of(int64_t M, int part, int parts) {
  const int64_t per = ((M + parts - 1) / parts + kActWarps - 1) / kActWarps * kActWarps;
  const int64_t from = part * per;
  return Rows{from, from + per < M ? from + per : M};
}

constexpr int kAtOnce = 2;   // rows whose loads a warp has under way

template <typename T, bool FP8>
__global__ void __launch_bounds__(kActThreads) act_backward_kernel(const __grid_constant__ FfnActArgs a, int parts) {
  __shared__ float sums[kActWarps][kActStrip];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = static_cast<int>(a.N), first = static_cast<int>(blockIdx.x) * kActStrip, c = first + lane * 8;
  const bool vec = a.vec;
  const Rows in = rows_of(a.M, blockIdx.y, parts);
  const bool act = a.act != GP_ACT_NONE;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  for (int64_t r0 = in.from + warp; r0 < in.to; r0 += kAtOnce * kActWarps) {
    Raw8<T> dy[kAtOnce];
    Kept<T, FP8> z[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r >= in.to) break;
      load8(dy[u], static_cast<const T*>(a.dy) + r * a.ld_dy, c, cols, vec);
      if (act) load_kept<T, FP8>(z[u], a.z[0], a.ldz[0], a.codes[0], r, c, cols, vec);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r >= in.to) break;
      float v[8], d[8];
      unpack8(dy[u], v);
      if (act) {
        float y[8];
        widen_kept<T, FP8>(y, z[u], a.e5m2);
        slopes(y, d, a.act);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= d[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
      if (a.dz[0]) {
        Raw8<T> o;
        pack8(v, o);
        store8(static_cast<T*>(a.dz[0]) + r * a.ld_dz[0], o, c, cols, vec);
      }
    }
  }
  if (!a.dbias) return;
  const Eight e = eight_columns(c, vec);
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[warp][e.first + i * e.stride - first] = sum[i];
  __syncthreads();
  const int col = first + static_cast<int>(threadIdx.x);
  if (col >= cols) return;
  float total = 0.f;
#pragma unroll
  for (int w = 0; w < kActWarps; ++w) total += sums[w][threadIdx.x];
  (parts > 1 ? a.partials + static_cast<int64_t>(blockIdx.y) * cols : a.dbias)[col] = total;
}

// dbias = sum of the parts, in their order.
__global__ void __launch_bounds__(kActThreads) sum_parts_kernel(const float* partials, float* dbias, int64_t N, int parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kActThreads + threadIdx.x;
  if (c >= N) return;
  float total = 0.f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) total += partials[p * N + c];
  dbias[c] = total;
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(kActThreads) gated_backward_kernel(const __grid_constant__ FfnActArgs a, int parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = static_cast<int>(a.N), c = static_cast<int>(blockIdx.x) * kActStrip + lane * 8;
  const bool vec = a.vec;
  const Rows in = rows_of(a.M, blockIdx.y, parts);
  for (int64_t r0 = in.from + warp; r0 < in.to; r0 += kAtOnce * kActWarps) {
    Raw8<T> dh[kAtOnce];
    Kept<T, FP8> kg[kAtOnce], ku[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r >= in.to) break;
      load8(dh[u], static_cast<const T*>(a.dy) + r * a.ld_dy, c, cols, vec);
      load_kept<T, FP8>(kg[u], a.z[0], a.ldz[0], a.codes[0], r, c, cols, vec);
      load_kept<T, FP8>(ku[u], a.z[1], a.ldz[1], a.codes[1], r, c, cols, vec);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r >= in.to) break;
      float v[8], g[8], d[8], up[8], t[8];
      unpack8(dh[u], v);
      widen_kept<T, FP8>(g, kg[u], a.e5m2);
      widen_kept<T, FP8>(up, ku[u], a.e5m2);
      slopes(g, d, a.act);
      Raw8<T> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] * up[i] * d[i];
      pack8(t, o);
      store8(static_cast<T*>(a.dz[0]) + r * a.ld_dz[0], o, c, cols, vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i] * g[i];
      pack8(t, o);
      store8(static_cast<T*>(a.dz[1]) + r * a.ld_dz[1], o, c, cols, vec);
      if (a.h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = g[i] * up[i];
        pack8(t, o);
        store8(static_cast<T*>(a.h) + r * a.ldh, o, c, cols, vec);
      }
    }
  }
}

__global__ void __launch_bounds__(256) pack_kernel(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst,
                                                   int64_t rows, int64_t cols) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = (cols + 7) / 8, n = rows * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / per, c = (i - r * per) * 8;
    const uint16_t* p = src + r * ld_src + c;
    uint16_t* o = dst + r * ld_dst + c;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < cols ? p[2 * j] : 0u, hi = c + 2 * j + 1 < cols ? p[2 * j + 1] : 0u;
      w[j] = lo | (hi << 16);
    }
    if (c + 8 <= cols) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) o[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

}  // namespace

int64_t ffn_act_parts(int64_t M, int64_t N, int sm_count) {
  // four blocks for each SM, and a row or two for each warp at least
  const int64_t strips = (N + kActStrip - 1) / kActStrip, most = (M + 2 * kActWarps - 1) / (2 * kActWarps);
  return std::max<int64_t>(1, std::min(most, (4 * sm_count + strips - 1) / strips));
}

namespace {

template <typename Kernel>
cudaError_t launch_act(Kernel k, const FfnActArgs& a, int parts, cudaStream_t stream, const void** kernel, gp_plan* plan) {
  *kernel = reinterpret_cast<const void*>(k);
  const dim3 grid(static_cast<unsigned>((a.N + kActStrip - 1) / kActStrip), static_cast<unsigned>(parts));
  plan->threads = kActThreads;
  plan->grid = static_cast<int32_t>(grid.x * grid.y);
  return launch_dependent(k, grid, dim3(kActThreads), 0, stream, a, parts);
}

}  // namespace

cudaError_t launch_ffn_act_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                    gp_plan* plan) {
  const int parts = static_cast<int>(ffn_act_parts(a.M, a.N, sm_count));
  plan->dtype = GP_PLAN_FFN;
  plan->kernel = "ffn_act_backward";
  const bool bf16 = a.type == GP_REAL_BF16, codes = a.codes[0].data != nullptr;
  const cudaError_t e =
      bf16 ? (codes ? launch_act(act_backward_kernel<__nv_bfloat16, true>, a, parts, stream, kernel, plan)
                    : launch_act(act_backward_kernel<__nv_bfloat16, false>, a, parts, stream, kernel, plan))
           : (codes ? launch_act(act_backward_kernel<__half, true>, a, parts, stream, kernel, plan)
                    : launch_act(act_backward_kernel<__half, false>, a, parts, stream, kernel, plan));
  if (e != cudaSuccess || !a.dbias || parts == 1) return e;
  return launch_dependent(sum_parts_kernel, dim3(static_cast<unsigned>((a.N + kActThreads - 1) / kActThreads)),
                          dim3(kActThreads), 0, stream, a.partials, a.dbias, a.N, parts);
}

cudaError_t launch_ffn_gated_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                      gp_plan* plan) {
  const int parts = static_cast<int>(ffn_act_parts(a.M, a.N, sm_count));
  plan->dtype = GP_PLAN_FFN;
  plan->kernel = "ffn_gated_backward";
  const bool bf16 = a.type == GP_REAL_BF16, codes = a.codes[0].data != nullptr;
  return bf16 ? (codes ? launch_act(gated_backward_kernel<__nv_bfloat16, true>, a, parts, stream, kernel, plan)
                       : launch_act(gated_backward_kernel<__nv_bfloat16, false>, a, parts, stream, kernel, plan))
              : (codes ? launch_act(gated_backward_kernel<__half, true>, a, parts, stream, kernel, plan)
                       : launch_act(gated_backward_kernel<__half, false>, a, parts, stream, kernel, plan));
}

cudaError_t launch_ffn_pack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols,
                            cudaStream_t stream, const void** kernel, gp_plan* plan) {
  const int64_t blocks = (rows * ((cols + 7) / 8) + 255) / 256;
  plan->dtype = GP_PLAN_FFN;
  plan->kernel = "ffn_pack_rows";
  plan->threads = 256;
  plan->grid = static_cast<int32_t>(std::min<int64_t>(blocks, 152 * 16));
  *kernel = reinterpret_cast<const void*>(pack_kernel);
  return launch_dependent(pack_kernel, dim3(plan->grid), dim3(256), 0, stream, static_cast<const uint16_t*>(src), ld_src,
                          static_cast<uint16_t*>(dst), ld_dst, rows, cols);
}

}  // namespace gp
