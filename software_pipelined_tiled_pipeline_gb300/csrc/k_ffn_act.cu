// k_ffn_act.cu -- the element-by-element part of the backward pass, and rows
// laid out for the tensor cores.
//
//   linear: dz = dy * act'(z), dbias = column sums of dz before its rounding
//   gated:  dg = dh * u * act'(g), du = dh * act(g), h = act(g) * u
//
// z, g and u come in 16 bits or as 8-bit codes with a scale for each row's 128
// values.  A block takes a strip of 128 columns (one group of codes per row) and a
// part of the rows, a warp every eighth of these, a lane four columns.  The bias
// gradient is summed in FP32 per lane, over the block's warps, over the up to eight
// parts of a cluster and, by a second kernel, over the clusters, each in a fixed
// order.  HBM bounds it: two bytes in and out per value, one for each 8-bit one.  Four values per lane and three rows under
// way keep it within 64 registers, so 48 KB of loads are under way on an SM (with
// eight values it took 255, and 4096 x 8192 with codes 111 us).
#include <algorithm>
#include "ffn_math.cuh"
#include "fp8_rows.cuh"

namespace gp {
namespace {

constexpr int kActThreads = 256, kActWarps = 8, kActStrip = 128;
constexpr int kAtOnce = 3;   // rows whose loads a warp has under way

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

// A lane's four columns of its strip: side by side where rows are on 16-byte
// boundaries, else every 32nd, so that a warp reads neighbouring values either way.
// All four exist with VEC; a block's last strip and rows off 16-byte boundaries go without.
template <bool VEC>
struct Four {
  int first, stride, cols;   // columns c = first + i * stride; `cols` there are
  __device__ __forceinline__ bool has(int i) const { return first + i * stride < cols; }
};

template <typename T, bool VEC>
__device__ __forceinline__ uint2 load4(const T* row, const Four<VEC>& f) {
  if (VEC) return *reinterpret_cast<const uint2*>(row + f.first);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f.has(i) ? reinterpret_cast<const uint16_t*>(row)[f.first + i * f.stride] : 0u;
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
template <typename T>
__device__ __forceinline__ void unpack4(float (&v)[4], uint2 w) {
  v[0] = word_lo<T>(w.x);
  v[1] = word_hi<T>(w.x);
  v[2] = word_lo<T>(w.y);
  v[3] = word_hi<T>(w.y);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store4(T* row, const float (&v)[4], const Four<VEC>& f) {
  T t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) from_f32(v[i], t[i]);
  if (VEC) {
    uint2 w;
    memcpy(&w, t, 8);
    *reinterpret_cast<uint2*>(row + f.first) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (f.has(i)) row[f.first + i * f.stride] = t[i];
}

// Four kept values of a row, as they lie in memory and as FP32.
template <typename T, bool FP8>
struct Kept {
  uint2 w;               // FP8: the codes, and their scale
};
template <typename T, bool FP8, bool VEC>
__device__ __forceinline__ Kept<T, FP8> load_kept(const void* z, int64_t ldz, const FfnCodes& q, int64_t row, int strip,
                                                  const Four<VEC>& f) {
  Kept<T, FP8> k;
  if constexpr (FP8) {
    const uint8_t* p = q.data + row * q.ld;
    k.w.y = __float_as_uint(q.scales[row * q.stride_row + strip * q.stride_col]);
    if (VEC) {
      k.w.x = *reinterpret_cast<const uint32_t*>(p + f.first);
    } else {
      k.w.x = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (f.has(i)) k.w.x |= static_cast<uint32_t>(p[f.first + i * f.stride]) << (8 * i);
    }
  } else {
    k.w = load4(static_cast<const T*>(z) + row * ldz, f);
  }
  return k;
}
template <typename T, bool FP8>
__device__ __forceinline__ void widen_kept(float (&v)[4], const Kept<T, FP8>& k, bool e5m2) {
  if constexpr (FP8) {
    const float scale = __uint_as_float(k.w.y);
    const float2 a = decode2(k.w.x, e5m2), b = decode2(k.w.x >> 16, e5m2);
    v[0] = a.x * scale;
    v[1] = a.y * scale;
    v[2] = b.x * scale;
    v[3] = b.y * scale;
  } else {
    unpack4<T>(v, k.w);
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

template <bool VEC>
__device__ __forceinline__ Four<VEC> columns_of(const FfnActArgs& a, int strip, int lane) {
  return Four<VEC>{strip * kActStrip + (VEC ? 4 * lane : lane), VEC ? 1 : 32, static_cast<int>(a.N)};
}

template <typename T, bool FP8, int ACT, bool VEC>
__device__ __forceinline__ void act_backward_rows(const FfnActArgs& a, const Rows& in, int strip, const Four<VEC>& f, int warp,
                                                  float (&sum)[4]) {
  constexpr int AT_ONCE = VEC ? kAtOnce : 1;
  for (int64_t r0 = in.from + warp; r0 < in.to; r0 += AT_ONCE * kActWarps) {
    uint2 dy[AT_ONCE];
    Kept<T, FP8> z[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r < in.to) {
        dy[u] = load4(static_cast<const T*>(a.dy) + r * a.ld_dy, f);
        if (ACT != GP_ACT_NONE) z[u] = load_kept<T, FP8, VEC>(a.z[0], a.ldz[0], a.codes[0], r, strip, f);
      }
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r < in.to) {
        float v[4];
        unpack4<T>(v, dy[u]);
        if (ACT != GP_ACT_NONE) {
          float y[4];
          widen_kept<T, FP8>(y, z[u], a.e5m2);
          ActSlope s[4];
          activate_slopes<ACT>(s, y);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] *= s[i].d;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[i];
        if (a.dz[0]) store4(static_cast<T*>(a.dz[0]) + r * a.ld_dz[0], v, f);
      }
    }
  }
}

#define GP_ACT_SWITCH(act, CALL)                            \
  switch (act) {                                            \
    case GP_ACT_RELU: CALL(GP_ACT_RELU); break;             \
    case GP_ACT_GELU: CALL(GP_ACT_GELU); break;             \
    case GP_ACT_GELU_TANH: CALL(GP_ACT_GELU_TANH); break;   \
    case GP_ACT_SILU: CALL(GP_ACT_SILU); break;             \
    case GP_ACT_SIGMOID: CALL(GP_ACT_SIGMOID); break;       \
    default: CALL(GP_ACT_NONE); break;                      \
  }

template <typename T, bool FP8>
__global__ void __launch_bounds__(kActThreads, 4) act_backward_kernel(const __grid_constant__ FfnActArgs a, int parts, int cluster) {
  __shared__ float sums[kActWarps][kActStrip];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, strip = blockIdx.x;
  const Rows in = rows_of(a.M, blockIdx.y, parts);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  const bool vec = a.vec && (strip + 1) * kActStrip <= a.N;
  if (vec) {
    const Four<true> f = columns_of<true>(a, strip, lane);
#define GP_CALL(ACT) act_backward_rows<T, FP8, ACT>(a, in, strip, f, warp, sum)
    GP_ACT_SWITCH(a.act, GP_CALL)
  } else {
    const Four<false> f = columns_of<false>(a, strip, lane);
    GP_ACT_SWITCH(a.act, GP_CALL)
#undef GP_CALL
  }
  if (!a.dbias) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[warp][vec ? 4 * lane + i : lane + 32 * i] = sum[i];
  __syncthreads();
  const int at = static_cast<int>(threadIdx.x), col = strip * kActStrip + at;
  float total = 0.f;
  if (at < kActStrip) {
#pragma unroll
    for (int w = 0; w < kActWarps; ++w) total += sums[w][at];
    sums[0][at] = total;
  }
  if (cluster > 1) {
    // the cluster's first block adds up what the others hold
    __syncwarp();
    cluster_sync();
    if (cluster_ctarank() == 0 && at < kActStrip) {
      for (int r = 1; r < cluster; ++r) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(smem_u32(&sums[0][at]), r)) : "memory");
        total += x;
      }
    }
    __syncwarp();
    cluster_sync();   // nobody leaves before its sums are read
    if (cluster_ctarank() != 0) return;
  }
  if (at >= kActStrip || col >= a.N) return;
  (parts > cluster ? a.partials + static_cast<int64_t>(blockIdx.y / cluster) * a.N : a.dbias)[col] = total;
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

template <typename T, bool FP8, int ACT, bool VEC>
__device__ __forceinline__ void gated_backward_rows(const FfnActArgs& a, const Rows& in, int strip, const Four<VEC>& f, int warp) {
  constexpr int AT_ONCE = VEC ? kAtOnce : 1;
  for (int64_t r0 = in.from + warp; r0 < in.to; r0 += AT_ONCE * kActWarps) {
    uint2 dh[AT_ONCE];
    Kept<T, FP8> kg[AT_ONCE], ku[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r < in.to) {
        dh[u] = load4(static_cast<const T*>(a.dy) + r * a.ld_dy, f);
        kg[u] = load_kept<T, FP8, VEC>(a.z[0], a.ldz[0], a.codes[0], r, strip, f);
        ku[u] = load_kept<T, FP8, VEC>(a.z[1], a.ldz[1], a.codes[1], r, strip, f);
      }
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int64_t r = r0 + u * kActWarps;
      if (r < in.to) {
        float v[4], g[4], up[4], dg[4], du[4], h[4];
        unpack4<T>(v, dh[u]);
        widen_kept<T, FP8>(g, kg[u], a.e5m2);
        widen_kept<T, FP8>(up, ku[u], a.e5m2);
        ActSlope s[4];
        activate_slopes<ACT>(s, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dg[i] = v[i] * up[i] * s[i].d;
          du[i] = v[i] * s[i].a;
          h[i] = s[i].a * up[i];
        }
        store4(static_cast<T*>(a.dz[0]) + r * a.ld_dz[0], dg, f);
        store4(static_cast<T*>(a.dz[1]) + r * a.ld_dz[1], du, f);
        if (a.h) store4(static_cast<T*>(a.h) + r * a.ldh, h, f);
      }
    }
  }
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(kActThreads, 4) gated_backward_kernel(const __grid_constant__ FfnActArgs a, int parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, strip = blockIdx.x;
  const Rows in = rows_of(a.M, blockIdx.y, parts);
  if (a.vec && (strip + 1) * kActStrip <= a.N) {
    const Four<true> f = columns_of<true>(a, strip, lane);
#define GP_CALL(ACT) gated_backward_rows<T, FP8, ACT>(a, in, strip, f, warp)
    GP_ACT_SWITCH(a.act, GP_CALL)
  } else {
    const Four<false> f = columns_of<false>(a, strip, lane);
    GP_ACT_SWITCH(a.act, GP_CALL)
#undef GP_CALL
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

namespace {

// Parts of the rows, with two rows for each warp at least.  Of one to four rounds of blocks (four on an SM) the one whose
// busiest SM has the fewest rows: 4096 x 8192 in 16 parts, 1.7 rounds, took 60 us, in 19, two rounds, 53.  With `groups`
// a power of two up to eight, or a multiple of eight, so that clusters of up to eight share them.
int64_t row_parts(int64_t M, int64_t N, int sm_count, bool groups) {
  const int64_t strips = (N + kActStrip - 1) / kActStrip, most = (M + 2 * kActWarps - 1) / (2 * kActWarps);
  const int64_t slots = 4 * static_cast<int64_t>(sm_count);
  int64_t best = 1, rows = 0;
  for (int64_t round = 1; round <= 4; ++round) {
    int64_t p = std::max<int64_t>(1, std::min(most, round * slots / strips));
    if (groups) p = p >= 8 ? p / 8 * 8 : (p >= 4 ? 4 : (p >= 2 ? 2 : 1));
    const int64_t per = ((M + p - 1) / p + kActWarps - 1) / kActWarps * kActWarps;
    const int64_t busiest = (strips * p + slots - 1) / slots * per;
    if (rows == 0 || busiest < rows) {
      best = p;
      rows = busiest;
    }
  }
  return best;
}

template <typename Kernel, typename... Args>
cudaError_t launch_act(Kernel k, const FfnActArgs& a, int parts, int cluster, cudaStream_t stream, const void** kernel,
                       gp_plan* plan, Args... args) {
  *kernel = reinterpret_cast<const void*>(k);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + kActStrip - 1) / kActStrip), static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kActThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  plan->threads = kActThreads;
  plan->grid = static_cast<int32_t>(cfg.gridDim.x * cfg.gridDim.y);
  return cudaLaunchKernelEx(&cfg, k, a, parts, args...);
}

}  // namespace

int64_t ffn_act_parts(int64_t M, int64_t N, int sm_count) {
  const int64_t parts = row_parts(M, N, sm_count, true);
  return parts > 8 ? parts / 8 : 1;
}

cudaError_t launch_ffn_act_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                    gp_plan* plan) {
  const int parts = static_cast<int>(row_parts(a.M, a.N, sm_count, a.dbias != nullptr)), cluster = a.dbias ? std::min(parts, 8) : 1;
  plan->dtype = GP_PLAN_FFN;
  plan->kernel = "ffn_act_backward";
  plan->k_splits = cluster;
  const bool bf16 = a.type == GP_REAL_BF16, codes = a.codes[0].data != nullptr;
  const cudaError_t e =
      bf16 ? (codes ? launch_act(act_backward_kernel<__nv_bfloat16, true>, a, parts, cluster, stream, kernel, plan, cluster)
                    : launch_act(act_backward_kernel<__nv_bfloat16, false>, a, parts, cluster, stream, kernel, plan, cluster))
           : (codes ? launch_act(act_backward_kernel<__half, true>, a, parts, cluster, stream, kernel, plan, cluster)
                    : launch_act(act_backward_kernel<__half, false>, a, parts, cluster, stream, kernel, plan, cluster));
  if (e != cudaSuccess || !a.dbias || parts <= 8) return e;
  return launch_dependent(sum_parts_kernel, dim3(static_cast<unsigned>((a.N + kActThreads - 1) / kActThreads)),
                          dim3(kActThreads), 0, stream, a.partials, a.dbias, a.N, parts / 8);
}

cudaError_t launch_ffn_gated_backward(const FfnActArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                      gp_plan* plan) {
  const int parts = static_cast<int>(row_parts(a.M, a.N, sm_count, false));
  plan->dtype = GP_PLAN_FFN;
  plan->kernel = "ffn_gated_backward";
  const bool bf16 = a.type == GP_REAL_BF16, codes = a.codes[0].data != nullptr;
  return bf16 ? (codes ? launch_act(gated_backward_kernel<__nv_bfloat16, true>, a, parts, 1, stream, kernel, plan)
                       : launch_act(gated_backward_kernel<__nv_bfloat16, false>, a, parts, 1, stream, kernel, plan))
              : (codes ? launch_act(gated_backward_kernel<__half, true>, a, parts, 1, stream, kernel, plan)
                       : launch_act(gated_backward_kernel<__half, false>, a, parts, 1, stream, kernel, plan));
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
