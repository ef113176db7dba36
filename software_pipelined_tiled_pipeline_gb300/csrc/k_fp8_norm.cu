// k_fp8_norm.cu -- RMS norm with the residual's addition and an 8-bit output,
// and its gradient.
//
//   h = round(x + residual),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight
//   g = dy * weight,  dx = rstd * (g - h * rstd * mean(g * h * rstd)) + dres,  dw = sum_rows dy * h * rstd
//
// Each input is read once and each output written once (the gradient of few
// rows reads dy and h twice).  A row stays in the registers of its threads (NCH
// chunks of 8 values each) from the load to the store, so the sum over the row
// costs one exchange between warps and no second read.  Chunk i of thread t holds columns
// 8 (i * threads + t) .., so a group of 128 columns is 16 neighbouring lanes
// and its maximum four shuffles.  Rows too long for the registers
// (kRowsMaxCols) are read twice.  Measured (BF16): the norm of 4096 x 8192 with
// a residual 46 us, 5.1 TB/s, 73 % of the issue slots (37 instructions per
// value); the gradient of 8192 x 8192 91 us, 5.9 TB/s, bound by HBM.
#include <cstring>
#include "fp8_rows.cuh"

namespace gp {
namespace {

constexpr int kLongThreads = 1024;
constexpr int kMaxChunks = 4;
// Threads of a block that holds NCH chunks per thread: with 512, a thread may
// use 128 registers.
template <int NCH>
constexpr int kRowThreads = NCH == 1 ? 256 : 512;
constexpr int64_t kRowsMaxCols = int64_t(kRowThreads<kMaxChunks>) * kMaxChunks * 8;   // 16384

// Sum over the threads of one row: blockDim.x threads, blockDim.y rows side by
// side.  `slots` holds two sets of 32 floats, used in turn, so one barrier per
// sum is enough.
__device__ __forceinline__ float row_sum(float v, float* slots) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5;
  float* mine = slots + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[warp] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < warps ? mine[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// Largest magnitude of eight values of each of the 16 lanes of a group.
__device__ __forceinline__ uint32_t group_max(const float (&y)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, abs_bits(y[k]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}
__device__ __forceinline__ void write_codes(uint8_t* row, const float (&y)[8], float inv, const NormArgs& a, int c) {
  uint2 w;
  if (a.e5m2) {
    w.x = fp8x4<true>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    w.y = fp8x4<true>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
  } else {
    w.x = fp8x4<false>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    w.y = fp8x4<false>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
  }
  store_codes8(row, w, c, static_cast<int>(a.cols), a.vec != 0);
}
// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Each block takes every gridDim.x-th row (or group of blockDim.y rows); the
// next row's loads are under way while this one is reduced and written.  h is
// kept as it is stored, and the weight is read again for each row (from the L1
// cache) where keeping it would cost the second block on an SM.
template <typename T, int NCH>
constexpr int kForwardBlocks = NCH == 1 ? 4 : (sizeof(T) == 2 && NCH == 2 ? 2 : 1);   // per SM
template <typename T, int NCH>
__global__ void __launch_bounds__(kRowThreads<NCH>, kForwardBlocks<T, NCH>)
    rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float slots[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const bool vec = a.vec != 0;
  const int lane = threadIdx.x & 31;
  const int cols = static_cast<int>(a.cols);
  const int col0 = threadIdx.x * 8, chunk = blockDim.x * 8;    // column of chunk i: col0 + i * chunk
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  constexpr bool KEEP_W = NCH == 1;
  float w[8];
  if (KEEP_W) load8_any(w, a.weight, a.weight_type, col0, cols, vec, a.vec_w != 0);
  Raw8<T> rx[NCH], rr[NCH];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = static_cast<const T*>(a.residual) + row * a.ld_res;
    const int n = row < a.rows ? cols : 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      load8(rx[i], x, col0 + i * chunk, n, vec);
      if (a.residual) load8(rr[i], r, col0 + i * chunk, n, vec);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  fetch(row);
  int set = 0;
  // (a block's spare rows take part in its barriers)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * blockDim.y; base < a.rows; base += step, row += step, set ^= 1) {
    const bool live = row < a.rows;
    Raw8<T> h[NCH];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float v[8];
      unpack8(rx[i], v);
      h[i] = rx[i];
      if (a.residual) {
        float r[8];
        unpack8(rr[i], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += r[k];
        pack8(v, h[i]);
        unpack8(h[i], v);               // the norm is of the rounded sum
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
    }
    fetch(row + step);
    if (a.h && live) {
      T* to = static_cast<T*>(a.h) + row * a.ld_h;
#pragma unroll
      for (int i = 0; i < NCH; ++i) store8(to, h[i], col0 + i * chunk, cols, vec);
    }
    ss = row_sum(ss, slots[set]);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (a.rstd && live && threadIdx.x == 0) a.rstd[row] = rstd;
    // y, the group maxima of all chunks, then their scales: the two divisions of
    // a scale are made once for two chunks, by half of a group's lanes each.
    float y[NCH][8];
    uint32_t most[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int col = col0 + i * chunk;
      if (!KEEP_W) load8_any(w, a.weight, a.weight_type, col, cols, vec, a.vec_w != 0);
      unpack8(h[i], y[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[i][k] = y[i][k] * rstd * w[k];
      if (a.y && live) {
        Raw8<T> ry;
        pack8(y[i], ry);
        store8(static_cast<T*>(a.y) + row * a.ld_y, ry, col, cols, vec);
      }
      if (a.q.data) most[i] = group_max(y[i]);
    }
    if (!a.q.data) continue;
    uint8_t* to = static_cast<uint8_t*>(a.q.data) + row * a.q.ld;
    float* scales = a.q.scales + row * a.q.stride_row;
    constexpr int PAIRS = NCH > 1 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < NCH; i += PAIRS) {
      const bool second = PAIRS == 2 && (lane & 8);
      const GroupScale g = group_scale(second ? most[i + PAIRS - 1] : most[i], a.fmax);
      const int col = col0 + (i + (second ? 1 : 0)) * chunk;
      // (the group's first column is inside the row exactly if the group has a scale)
      if ((lane & (PAIRS == 2 ? 7 : 15)) == 0 && live && (col & ~127) < a.cols)
        scales[(col >> 7) * a.q.stride_col] = g.scale;
#pragma unroll
      for (int u = 0; u < PAIRS; ++u) {
        const float inv = PAIRS == 2 ? __shfl_sync(0xffffffffu, g.inv, (lane & 16) + 8 * u) : g.inv;
        if (live) write_codes(to, y[i + u], inv, a, col0 + (i + u) * chunk);
      }
    }
  }
}

// Rows longer than kRowsMaxCols: one block per row, two passes over it (2048 x
// 32768 with a residual, BF16 159 us, FP32 192 us: 3.0 and 4.5 TB/s of what has to
// move; one row of 20480 6.9 us).  The
// second pass takes h from where the first stored it (x or the residual may be
// that place), else forms it again.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_long_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float slots[32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const bool vec = a.vec != 0;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const int lane = threadIdx.x & 31;
  const int cols = static_cast<int>(a.cols), step = blockDim.x * 8;
  const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* const res = static_cast<const T*>(a.residual) + row * a.ld_res;
  T* const to = static_cast<T*>(a.h) + row * a.ld_h;
  auto form = [&](int c, Raw8<T>& raw, float (&h)[8]) {
    load8(raw, x, c, cols, vec);
    unpack8(raw, h);
    if (!a.residual) return;
    float r[8];
    load8(raw, res, c, cols, vec);
    unpack8(raw, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] += r[k];
    pack8(h, raw);
    unpack8(raw, h);
  };
  // (whole groups of 128 columns: with rows off their alignment the last one's lanes each hold some of it)
  const int64_t end = (a.cols + 127) / 128 * 128;
  float ss = 0.f;
  for (int64_t at = threadIdx.x * 8; at < end; at += step) {
    const int c = static_cast<int>(at);
    Raw8<T> raw;
    float h[8];
    form(c, raw, h);
    if (a.h) store8(to, raw, c, cols, vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(h[k], h[k], ss);
  }
  ss = row_sum(ss, slots);
  const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  for (int64_t base = 0; base < end; base += step) {   // (whole blocks: the shuffles need every lane)
    const int64_t at = base + threadIdx.x * 8;
    const int n = at < end ? cols : 0;
    const int c = at < end ? static_cast<int>(at) : 0;
    Raw8<T> raw;
    float h[8], w[8];
    if (a.h) {
      load8(raw, to, c, n, vec);
      unpack8(raw, h);
    } else {
      form(c, raw, h);
    }
    load8_any(w, a.weight, a.weight_type, c, n, vec, a.vec_w != 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = h[k] * rstd * w[k];
    if (a.y) {
      pack8(w, raw);
      store8(static_cast<T*>(a.y) + row * a.ld_y, raw, c, n, vec);
    }
    if (!a.q.data) continue;
    const GroupScale g = group_scale(group_max(w), a.fmax);
    if (n == 0) continue;                              // (a whole group's lanes alike)
    if ((lane & 15) == 0) a.q.scales[row * a.q.stride_row + (c >> 7) * a.q.stride_col] = g.scale;
    write_codes(static_cast<uint8_t*>(a.q.data) + row * a.q.ld, w, g.inv, a, c);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A thread's eight column sums to its row of the partial sums.
__device__ __forceinline__ void store_sums(float* row, const float (&v)[8], int c, int cols, bool vec) {
  if (vec && cols % 4 == 0 && c + 8 <= cols) {
    reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  const Eight e = eight_columns(c, vec);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e.first + k * e.stride < cols) row[e.first + k * e.stride] = v[k];
}

// The weight's gradient of 64 columns, by one block: eight threads to a row,
// the rows dealt out among the rest of the block, whose sums meet in a fixed order.
constexpr int kStripCols = 64;
template <typename T>
__device__ __forceinline__ void column_sums(const NormGradArgs& a, float (*s)[kStripCols]) {
  const int t = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const int cols = static_cast<int>(a.cols), c = blockIdx.x * kStripCols + (t & 7) * 8;
  const bool vec = a.vec != 0;
  const int64_t step = threads >> 3;
  const Eight e = eight_columns(c, vec);
  float dw[8] = {};
  // A thread has `batch` rows under way together, and their loads carry no
  // branch: past the last row the thread's first one is read again and not
  // added, past the last column the first one is (those sums go nowhere).  whole:
  // the eight columns are one aligned run.
  auto walk = [&](auto whole, auto batch) {
    constexpr int BATCH = batch.value;
    for (int64_t row = t >> 3; row < a.rows; row += BATCH * step) {
      Raw8<T> rdy[BATCH], rh[BATCH];
      float rstd[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const bool in = row + u * step < a.rows;
        const int64_t at = in ? row + u * step : row;
        const T* dy = static_cast<const T*>(a.dy) + at * a.ld_dy;
        const T* h = static_cast<const T*>(a.h) + at * a.ld_h;
        if constexpr (whole.value) {
#pragma unroll
          for (int i = 0; i < Raw8<T>::WORDS; ++i) {
            rdy[u].w[i] = reinterpret_cast<const uint4*>(dy + c)[i];
            rh[u].w[i] = reinterpret_cast<const uint4*>(h + c)[i];
          }
        } else {
          T x[8], y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = e.first + k * e.stride < cols ? e.first + k * e.stride : e.first;
            x[k] = dy[col];
            y[k] = h[col];
          }
          memcpy(&rdy[u], x, sizeof(x));
          memcpy(&rh[u], y, sizeof(y));
        }
        rstd[u] = a.rstd[at];
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        float dy[8], h[8];
        unpack8(rdy[u], dy);
        unpack8(rh[u], h);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float p = dy[k] * (h[k] * rstd[u]);
          dw[k] += row + u * step < a.rows ? p : 0.f;
        }
      }
    }
  };
  // (threads past the row's end have nothing to add; the shuffles below need them)
  if (vec && c + 8 <= cols)
    walk(std::true_type(), std::integral_constant<int, 4>());
  else if (e.first < cols)
    walk(std::false_type(), std::integral_constant<int, 2>());
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], 8);
    dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], 16);
    if ((t & 31) < 8) s[t >> 5][t * 8 % kStripCols + k] = dw[k];
  }
  __syncthreads();
  if (t >= kStripCols) return;
  float v = s[0][t];
  for (int w = 1; w < threads >> 5; ++w) v += s[w][t];
  const Eight own = eight_columns(blockIdx.x * kStripCols + (t & ~7), vec);
  const int col = own.first + (t & 7) * own.stride;
  if (col < cols) a.dw[col] = v;
}

// Each block takes every gridDim.x-th row (or group of blockDim.y rows).  The
// weight's gradient needs no sum over a row, as rstd is given, so with few rows
// the first col_blocks blocks work it out by columns, reading dy and h a second
// time (from L2): one launch and no workspace.  With more rows each block keeps
// its columns' share in registers, and sum_parts_kernel adds the shares in order.
template <typename T, int NCH>
__global__ void __launch_bounds__(kRowThreads<NCH>) rmsnorm_grad_kernel(const __grid_constant__ NormGradArgs a) {
  __shared__ float slots[2][32];
  __shared__ float strip[kRowThreads<NCH> / 32][kStripCols];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x < static_cast<unsigned>(a.col_blocks)) {
    column_sums<T>(a, strip);
    return;
  }
  const int block = blockIdx.x - a.col_blocks, blocks = gridDim.x - a.col_blocks;
  const bool vec = a.vec != 0;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  // The weight of up to two chunks stays in registers; with four, each row reads
  // it again from the L1 cache.  (512 threads have 128 registers each: four chunks
  // spill all the same, 180 bytes stored per thread in 16-bit types and 292 in
  // FP32, and so do two of FP32, 92 bytes.)
  constexpr bool KEEP_W = NCH <= 2;
  const int cols = static_cast<int>(a.cols);
  const int col0 = threadIdx.x * 8, chunk = blockDim.x * 8;    // column of chunk i: col0 + i * chunk
  float w[KEEP_W ? NCH : 1][8], dw[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if (KEEP_W) load8_any(w[KEEP_W ? i : 0], a.weight, a.weight_type, col0 + i * chunk, cols, vec, a.vec_w != 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.f;
  }
  // The next row's values come while this one is reduced and written.
  constexpr bool AHEAD = NCH <= 2;
  Raw8<T> ndy[NCH], nh[NCH], nr[NCH];
  float nrstd = 0.f;
  auto fetch = [&](int64_t row) {
    const bool in = row < a.rows;
    const int n = in ? cols : 0;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const T* h = static_cast<const T*>(a.h) + row * a.ld_h;
    const T* r = static_cast<const T*>(a.dres) + row * a.ld_dres;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      load8(ndy[i], dy, col0 + i * chunk, n, vec);
      load8(nh[i], h, col0 + i * chunk, n, vec);
      if (a.dres) load8(nr[i], r, col0 + i * chunk, n, vec);
    }
    nrstd = in ? a.rstd[row] : 0.f;
  };
  const int64_t step = static_cast<int64_t>(blocks) * blockDim.y;
  int set = 0;
  if (AHEAD) fetch(static_cast<int64_t>(block) * blockDim.y + threadIdx.y);
  for (int64_t base = static_cast<int64_t>(block) * blockDim.y; base < a.rows; base += step, set ^= 1) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    if (!AHEAD) fetch(row);
    Raw8<T> rdy[NCH], rh[NCH], rr[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      rdy[i] = ndy[i];
      rh[i] = nh[i];
      rr[i] = nr[i];
    }
    const float rstd = nrstd;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int wi = KEEP_W ? i : 0;
      if (!KEEP_W)
        load8_any(w[0], a.weight, a.weight_type, col0 + i * chunk, cols, vec, a.vec_w != 0);
      float dy[8], h[8];
      unpack8(rdy[i], dy);
      unpack8(rh[i], h);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float unit = h[k] * rstd;
        const float p = dy[k] * unit;
        dw[i][k] += p;
        sum = fmaf(p, w[wi][k], sum);
      }
    }
    if (AHEAD) fetch(row + step);
    const float mean = row_sum(sum, slots[set]) * inv_cols;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int col = col0 + i * chunk;
      const int wi = KEEP_W ? i : 0;
      if (!KEEP_W) load8_any(w[0], a.weight, a.weight_type, col, cols, vec, a.vec_w != 0);
      float dy[8], h[8], o[8];
      unpack8(rdy[i], dy);
      unpack8(rh[i], h);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = rstd * (dy[k] * w[wi][k] - h[k] * rstd * mean);
      if (a.dres) {
        float r[8];
        unpack8(rr[i], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += r[k];
      }
      Raw8<T> out;
      pack8(o, out);
      store8(static_cast<T*>(a.dx) + row * a.ld_dx, out, col, cols, vec);
    }
  }
  if (!a.partials) return;
  float* part = a.partials + (static_cast<int64_t>(block) * blockDim.y + threadIdx.y) * a.cols;
#pragma unroll
  for (int i = 0; i < NCH; ++i) store_sums(part, dw[i], col0 + i * chunk, cols, vec);
}

// Rows longer than kRowsMaxCols: dx in two passes over the row, dw by columns
// (2048 x 32768, BF16 207 us, FP32 295 us: 2.6 and 3.6 TB/s, as dy and h are read
// three times; one row of 20480 8.4 us).
template <typename T>
__global__ void __launch_bounds__(kLongThreads) rmsnorm_grad_long_kernel(const __grid_constant__ NormGradArgs a) {
  __shared__ float slots[32];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const bool vec = a.vec != 0;
  const float rstd = a.rstd[row];
  const int cols = static_cast<int>(a.cols), step = blockDim.x * 8;
  const int64_t end = (a.cols + 127) / 128 * 128;
  float sum = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    const float mean = pass ? row_sum(sum, slots) / static_cast<float>(a.cols) : 0.f;
    for (int64_t at = threadIdx.x * 8; at < end; at += step) {
      const int c = static_cast<int>(at);
      Raw8<T> raw;
      float dy[8], h[8], w[8];
      load8(raw, static_cast<const T*>(a.dy) + row * a.ld_dy, c, cols, vec);
      unpack8(raw, dy);
      load8(raw, static_cast<const T*>(a.h) + row * a.ld_h, c, cols, vec);
      unpack8(raw, h);
      load8_any(w, a.weight, a.weight_type, c, cols, vec, a.vec_w != 0);
      if (pass == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fmaf(dy[k] * (h[k] * rstd), w[k], sum);
        continue;
      }
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = rstd * (dy[k] * w[k] - h[k] * rstd * mean);
      if (a.dres) {
        float r[8];
        load8(raw, static_cast<const T*>(a.dres) + row * a.ld_dres, c, cols, vec);
        unpack8(raw, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += r[k];
      }
      pack8(o, raw);
      store8(static_cast<T*>(a.dx) + row * a.ld_dx, raw, c, cols, vec);
    }
  }
}

constexpr int kLongParts = 32;   // shares of the rows in the column sums of long rows

template <typename T>
__global__ void __launch_bounds__(256) rmsnorm_dw_long_kernel(const __grid_constant__ NormGradArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int cols = static_cast<int>(a.cols);
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 8;
  if (at >= (a.cols + 127) / 128 * 128) return;
  const int c = static_cast<int>(at);
  const int parts = gridDim.y;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += parts) {
    Raw8<T> raw;
    float dy[8], h[8];
    load8(raw, static_cast<const T*>(a.dy) + row * a.ld_dy, c, cols, a.vec != 0);
    unpack8(raw, dy);
    load8(raw, static_cast<const T*>(a.h) + row * a.ld_h, c, cols, a.vec != 0);
    unpack8(raw, h);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[k] += dy[k] * (h[k] * rstd);
  }
  store_sums(a.partials + static_cast<int64_t>(blockIdx.y) * a.cols, dw, c, cols, a.vec != 0);
}

// dw[c] = sum over parts of partials[part][c], in a fixed order: 8 threads per
// column take every eighth part each, then meet in shared memory.
constexpr int kSumCols = 32, kSumWays = 8;
__global__ void __launch_bounds__(kSumCols * kSumWays) sum_parts_kernel(const float* partials, float* dw, int64_t parts,
                                                                       int64_t cols) {
  __shared__ float s[kSumWays][kSumCols];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumCols + threadIdx.x;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t p = threadIdx.y; p < parts; p += kSumWays) v += partials[p * cols + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= cols) return;
#pragma unroll
  for (int k = 1; k < kSumWays; ++k) v += s[k][threadIdx.x];
  dw[c] = v;
}

__global__ void __launch_bounds__(256) fill_f32_kernel(float* p, int64_t n, float value) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p[i] = value;
}

// Threads per row, chunks per thread and rows per block for a row of `cols`.
struct RowShape {
  int threads, chunks, rows;
};
RowShape row_shape(int64_t cols) {
  RowShape s;
  const int64_t chunks = (cols + 127) / 128 * 16;   // (whole groups: see Eight)
  s.chunks = chunks <= kRowThreads<1> ? 1 : (chunks <= 2 * kRowThreads<2> ? 2 : 4);
  const int64_t per = (chunks + s.chunks - 1) / s.chunks;
  s.threads = static_cast<int>((per + 31) / 32 * 32);
  s.rows = s.threads >= 128 ? 1 : 128 / s.threads;
  return s;
}

// Blocks for `rows` rows, each looping over its own: what fits on the device at `per_sm` threads per SM.
constexpr int kBackwardThreads = 512;
int64_t row_blocks(int64_t rows, const RowShape& s, int sm_count, int per_sm) {
  const int64_t want = (rows + s.rows - 1) / s.rows;
  const int at_once = per_sm / (s.threads * s.rows);
  const int64_t most = static_cast<int64_t>(sm_count) * (at_once > 1 ? at_once : 1);
  return want < most ? want : most;
}

template <typename T>
cudaError_t forward_type(const NormArgs& a, int sm_count, cudaStream_t stream, const void** kernel, gp_plan* plan) {
  if (a.cols > kRowsMaxCols) {
    auto k = rmsnorm_long_kernel<T>;
    *kernel = reinterpret_cast<const void*>(k);
    plan->threads = kLongThreads;
    plan->grid = static_cast<int32_t>(a.rows);
    return launch_dependent(k, dim3(static_cast<unsigned>(a.rows)), dim3(kLongThreads), 0, stream, a);
  }
  const RowShape s = row_shape(a.cols);
  auto k = s.chunks == 1 ? rmsnorm_kernel<T, 1> : (s.chunks == 2 ? rmsnorm_kernel<T, 2> : rmsnorm_kernel<T, 4>);
  const int per_sm = s.chunks == 1 ? kForwardBlocks<T, 1> * kRowThreads<1>
                                   : (s.chunks == 2 ? kForwardBlocks<T, 2> * kRowThreads<2> : kRowThreads<4>);
  *kernel = reinterpret_cast<const void*>(k);
  plan->threads = s.threads * s.rows;
  plan->grid = static_cast<int32_t>(row_blocks(a.rows, s, sm_count, per_sm));
  return launch_dependent(k, dim3(static_cast<unsigned>(plan->grid)), dim3(s.threads, s.rows), 0, stream, a);
}

// Rows up to which the weight's gradient is worked out by columns (see
// rmsnorm_grad_kernel).  Measured against partial sums and their kernel, us of
// device time, columns | partials, 512 rows (a call saves 5 us of host time
// besides): BF16 64 columns 4.0 | 6.8, 512 4.3 | 7.2, 1000 5.4 | 7.8, 2056 6.3 | 9.0,
// 8192 10.0 | 11.9, 16384 21.1 | 24.2; FP32 64 4.6 | 6.1, 2056 9.3 | 12.4, 8192
// 17.6 | 18.7, 16384 40.9 | 42.5.  At 1024 rows of 16384 47.0 | 43.6 (FP32 84 | 72).
// With rows off 16-byte boundaries up to 200 rows (BF16 1001 columns 6.1 | 6.4, 65
// 4.6 | 5.1); at 512 rows 65 columns take 9.1 | 7.1, FP32 1001 11.3 | 7.4, as a call
// 16 | 21.  The alignment is no part of the rule: the workspace goes by sizes alone.
constexpr int64_t kFewRows = 512;
bool by_columns(int64_t rows, int64_t cols) { return rows <= kFewRows && cols <= kRowsMaxCols; }

bool overlap(const void* p, int64_t ld_p, const void* q, int64_t ld_q, const NormGradArgs& a) {
  const int w = real_bytes(a.type);
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return x < y + ((a.rows - 1) * ld_q + a.cols) * w && y < x + ((a.rows - 1) * ld_p + a.cols) * w;
}

template <typename T>
cudaError_t backward_type(NormGradArgs a, int sm_count, cudaStream_t stream, const void** kernel,
                          gp_plan* plan) {
  if (a.cols > kRowsMaxCols) {
    cudaError_t e;
    if (a.partials) {
      const int64_t chunks = (a.cols + 127) / 128 * 16;
      const dim3 grid(static_cast<unsigned>((chunks + 255) / 256),
                      static_cast<unsigned>(a.rows < kLongParts ? a.rows : kLongParts));
      if ((e = launch_dependent(rmsnorm_dw_long_kernel<T>, grid, dim3(256), 0, stream, a)) != cudaSuccess) return e;
    }
    auto k = rmsnorm_grad_long_kernel<T>;
    *kernel = reinterpret_cast<const void*>(k);
    plan->threads = kLongThreads;
    plan->grid = static_cast<int32_t>(a.rows);
    return launch_dependent(k, dim3(static_cast<unsigned>(a.rows)), dim3(kLongThreads), 0, stream, a);
  }
  const RowShape s = row_shape(a.cols);
  auto k = s.chunks == 1 ? rmsnorm_grad_kernel<T, 1>
                         : (s.chunks == 2 ? rmsnorm_grad_kernel<T, 2> : rmsnorm_grad_kernel<T, 4>);
  *kernel = reinterpret_cast<const void*>(k);
  plan->threads = s.threads * s.rows;
  plan->grid = static_cast<int32_t>(row_blocks(a.rows, s, sm_count, kBackwardThreads));
  if (a.dw && by_columns(a.rows, a.cols)) {
    a.col_blocks = static_cast<int32_t>((a.cols + 127) / 128 * (128 / kStripCols));
    if (overlap(a.dx, a.ld_dx, a.dy, a.ld_dy, a) || overlap(a.dx, a.ld_dx, a.h, a.ld_h, a)) {
      // in place: the columns are read before any row is written
      const cudaError_t e = launch_dependent(k, dim3(a.col_blocks), dim3(s.threads, s.rows), 0, stream, a);
      if (e != cudaSuccess) return e;
      a.col_blocks = 0;
    }
    plan->grid += a.col_blocks;
  }
  return launch_dependent(k, dim3(static_cast<unsigned>(plan->grid)), dim3(s.threads, s.rows), 0, stream, a);
}

}  // namespace

cudaError_t launch_fp8_rmsnorm(const NormArgs& a, int sm_count, cudaStream_t stream, const void** kernel, gp_plan* plan) {
  plan->kernel = "fp8_rmsnorm";
  switch (a.type) {
    case GP_REAL_F16: return forward_type<__half>(a, sm_count, stream, kernel, plan);
    case GP_REAL_BF16: return forward_type<__nv_bfloat16>(a, sm_count, stream, kernel, plan);
    default: return forward_type<float>(a, sm_count, stream, kernel, plan);
  }
}

cudaError_t launch_fp8_fill_f32(float* p, int64_t n, float value, cudaStream_t stream) {
  const int64_t blocks = (n + 255) / 256;
  return launch_dependent(fill_f32_kernel, dim3(static_cast<unsigned>(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream,
                          p, n, value);
}

int64_t fp8_rmsnorm_backward_parts(int64_t rows, int64_t cols, int sm_count) {
  if (by_columns(rows, cols)) return 0;
  if (cols > kRowsMaxCols) return rows < kLongParts ? rows : kLongParts;
  const RowShape s = row_shape(cols);
  return row_blocks(rows, s, sm_count, kBackwardThreads) * s.rows;
}

cudaError_t launch_fp8_rmsnorm_backward(const NormGradArgs& a, int sm_count, cudaStream_t stream, const void** kernel,
                                        gp_plan* plan) {
  plan->kernel = "fp8_rmsnorm_backward";
  if (a.rows == 0) return launch_fp8_fill_f32(a.dw, a.cols, 0.f, stream);
  cudaError_t e;
  switch (a.type) {
    case GP_REAL_F16: e = backward_type<__half>(a, sm_count, stream, kernel, plan); break;
    case GP_REAL_BF16: e = backward_type<__nv_bfloat16>(a, sm_count, stream, kernel, plan); break;
    default: e = backward_type<float>(a, sm_count, stream, kernel, plan); break;
  }
  if (e != cudaSuccess || !a.partials) return e;
  return launch_dependent(sum_parts_kernel, dim3(static_cast<unsigned>((a.cols + kSumCols - 1) / kSumCols)),
                          dim3(kSumCols, kSumWays), 0, stream, static_cast<const float*>(a.partials), a.dw,
                          fp8_rmsnorm_backward_parts(a.rows, a.cols, sm_count), a.cols);
}

}  // namespace gp
