// k_fp8_quant.cu -- quantisation of a 16- or 32-bit matrix to 8-bit floating
// point with one FP32 scale per 128 values of a row (and/or of a column, for
// the transpose) or per 128 x 128 block.
//
//   scale = max(amax / FMAX, 2^-64),  code = rne(x * (1 / scale))
//
// One CTA takes one 128 x 128 tile, so each group of 128 along a row, each
// along a column and each block lies in one CTA and x is read once for both
// outputs.  Thread t holds the 8 x 8 values of rows 8 (t / 16) .. and columns
// 8 (t % 16) ..: a row's 16 threads lie in half a warp (its maximum takes four
// shuffles), a row's codes leave as 128 contiguous bytes, and a column's eight
// codes are one 8-byte word of the transposed tile, which goes through shared
// memory so that it leaves in 128-byte rows as well.
#include <cstring>
#include "fp8_rows.cuh"

namespace gp {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;

struct QuantArgs {
  const void* x;
  int64_t ldx;
  int64_t rows, cols;
  gp_fp8_matrix q, qt;   // data NULL: not written
  int64_t tiles_c;       // tiles along the columns
  float fmax;
  int32_t e5m2;
};

// Codes of the thread's eight rows, 8 at a time along each row (c: the thread's columns in the tile's row r).
template <bool E5M2, bool VEC, typename T>
__device__ __forceinline__ void write_rows(const Raw8<T> (&v)[8], const float (&inv)[8], const QuantArgs& a,
                                           int64_t r, int64_t c0, int c, int rows_in, int cols_in, bool whole) {
  uint8_t* out = static_cast<uint8_t*>(a.q.data) + r * a.q.ld + c0;
#pragma unroll
  for (int i = 0; i < 8; ++i, out += a.q.ld) {
    if (!whole && i >= rows_in) break;
    const float f = inv[i];
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = value_of(v[i], k) * f;
    uint2 w;
    w.x = fp8x4<E5M2>(x[0], x[1], x[2], x[3]);
    w.y = fp8x4<E5M2>(x[4], x[5], x[6], x[7]);
    if (whole)
      *reinterpret_cast<uint2*>(out + c) = w;
    else
      store_codes8(out, w, c, cols_in, VEC);
  }
}

// The transposed tile in shared memory: 128 rows (x's columns) of 16 words of
// 8 bytes; word w of a row that belongs to thread k of its 16 lies at w ^ k, so
// that the 16 threads of half a warp (k = 0..15, one w) and the 8 readers of a
// row touch all banks once.
template <bool E5M2, typename T>
__device__ __forceinline__ void stage_columns(const Raw8<T> (&v)[8], const float* inv_col, uint2* tile, int rb, int cc, Eight e) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = e.first + j * e.stride;
    const float f = inv_col[col];
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = value_of(v[i], j) * f;
    uint2 w;
    w.x = fp8x4<E5M2>(x[0], x[1], x[2], x[3]);
    w.y = fp8x4<E5M2>(x[4], x[5], x[6], x[7]);
    tile[col * 16 + (rb ^ cc)] = w;
  }
}

// VEC: x's rows are on 16-byte boundaries.
template <typename T, bool BLOCKS, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) quantize_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ __align__(16) uint2 tile[kTile * 16];      // 16 KB
  __shared__ uint32_t part[8 * kTile];                  // per warp: column maxima (or one block maximum)
  __shared__ float inv_col[kTile];
  pdl_launch_dependents();
  pdl_wait();

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rb = t >> 4, cc = t & 15;
  const int64_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
  const int64_t r0 = tr * kTile, c0 = tc * kTile;
  const int64_t r = r0 + rb * 8;
  const int c = cc * 8;                                       // the thread's columns (see Eight) in the tile
  const Eight e = eight_columns(c, VEC);
  const int rows_in = static_cast<int>(a.rows - r < 0 ? 0 : (a.rows - r > 8 ? 8 : a.rows - r));
  const int cols_in = static_cast<int>(a.cols - c0 > kTile ? kTile : a.cols - c0);

  // The values stay as they came (16-bit ones two to a register), so that four
  // blocks of 16-bit tiles fit on an SM and its loads overlap their work.
  Raw8<T> v[8];
  const T* x = static_cast<const T*>(a.x) + r * a.ldx + c0;
  // (a whole tile's loads and stores carry no checks: every thread of the block takes the same way)
  const bool whole = VEC && a.rows - r0 >= kTile && cols_in == kTile;
  if (whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) load8(v[i], x + i * a.ldx, c, kTile, true);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) load8(v[i], x + i * a.ldx, c, i < rows_in ? cols_in : 0, VEC);
  }
  constexpr int WORDS = static_cast<int>(sizeof(T)) * 2;       // 32-bit words of eight values
  constexpr int PER = 8 / WORDS;                                // values per word
  auto word = [&](int i, int k) { return raw_abs<T>(reinterpret_cast<const uint32_t*>(&v[i])[k]); };
  auto widest = [&](uint32_t m) {                               // the larger of a word's magnitudes, as FP32 bits
    return PER == 1 ? m : max(raw_to_bits<T>(m, 0), raw_to_bits<T>(m, 1));
  };

  if (BLOCKS) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < WORDS; ++k) m = raw_max<T>(m, word(i, k));
    m = __reduce_max_sync(0xffffffffu, widest(m));
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, part[w]);
    const GroupScale g = group_scale(m, a.fmax);
    if (t == 0) {
      if (a.q.data) a.q.scales[tr * a.q.stride_row + tc * a.q.stride_col] = g.scale;
      if (a.qt.data) a.qt.scales[tc * a.qt.stride_row + tr * a.qt.stride_col] = g.scale;
    }
    if (a.q.data) {
      float inv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) inv[i] = g.inv;
      if (a.e5m2) write_rows<true, VEC>(v, inv, a, r, c0, c, rows_in, cols_in, whole);
      else write_rows<false, VEC>(v, inv, a, r, c0, c, rows_in, cols_in, whole);
    }
    if (!a.qt.data) return;
    if (t < kTile) inv_col[t] = g.inv;
  } else {
    if (a.qt.data) {
      // a warp's rows of each column: two half warps of eight rows each
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        uint32_t m = word(0, k);
#pragma unroll
        for (int i = 1; i < 8; ++i) m = raw_max<T>(m, word(i, k));
        m = raw_max<T>(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < 16) {
#pragma unroll
          for (int u = 0; u < PER; ++u) part[warp * kTile + e.first + (k * PER + u) * e.stride] = raw_to_bits<T>(m, u);
        }
      }
    }
    if (a.q.data) {
      float inv[8];
      // Thread cc of a row's 16 works out the scale of row cc mod 8 and the others take it from there.
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = word(i, 0);
#pragma unroll
        for (int k = 1; k < WORDS; ++k) m = raw_max<T>(m, word(i, k));
#pragma unroll
        for (int d = 1; d < 16; d *= 2) m = raw_max<T>(m, __shfl_xor_sync(0xffffffffu, m, d));
        if ((cc & 7) == i) most = m;
      }
      const GroupScale g = group_scale(widest(most), a.fmax);
#pragma unroll
      for (int i = 0; i < 8; ++i) inv[i] = __shfl_sync(0xffffffffu, g.inv, (lane & 16) + i);
      if (cc < rows_in) a.q.scales[(r + cc) * a.q.stride_row + tc * a.q.stride_col] = g.scale;   // (rows_in <= 8)
      if (a.e5m2) write_rows<true, VEC>(v, inv, a, r, c0, c, rows_in, cols_in, whole);
      else write_rows<false, VEC>(v, inv, a, r, c0, c, rows_in, cols_in, whole);
    }
    if (!a.qt.data) return;
    __syncthreads();
    if (t < kTile) {
      uint32_t m = part[t];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = max(m, part[w * kTile + t]);
      const GroupScale g = group_scale(m, a.fmax);
      inv_col[t] = g.inv;
      if (c0 + t < a.cols) a.qt.scales[(c0 + t) * a.qt.stride_row + tr * a.qt.stride_col] = g.scale;
    }
  }
  __syncthreads();
  if (a.e5m2) stage_columns<true>(v, inv_col, tile, rb, cc, e);
  else stage_columns<false>(v, inv_col, tile, rb, cc, e);
  __syncthreads();
  uint8_t* out = static_cast<uint8_t*>(a.qt.data);
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int idx = it * kThreads + t;
    const int col = idx >> 3, pair = idx & 7;          // 16 rows of x: words 2 pair and 2 pair + 1
    const int k = VEC ? col >> 3 : col & 15;        // the thread that holds it
    uint4 w = *reinterpret_cast<const uint4*>(&tile[col * 16 + ((2 * pair) ^ (k & 14))]);
    if (k & 1) w = make_uint4(w.z, w.w, w.x, w.y);
    const int64_t row = r0 + pair * 16;
    if (c0 + col >= a.cols || row >= a.rows) continue;
    uint8_t* p = out + (c0 + col) * a.qt.ld + row;
    if (row + 16 <= a.rows) {
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      const int left = static_cast<int>(a.rows - row);
      store_codes8(p, make_uint2(w.x, w.y), 0, left, true);
      store_codes8(p, make_uint2(w.z, w.w), 8, left, true);
    }
  }
}

template <typename T>
cudaError_t launch_type(const QuantArgs& a, bool blocks, int64_t tiles, cudaStream_t stream, const void** kernel) {
  const bool vec = vec16(a.x, a.ldx, sizeof(T));
  auto k = blocks ? (vec ? quantize_kernel<T, true, true> : quantize_kernel<T, true, false>)
                  : (vec ? quantize_kernel<T, false, true> : quantize_kernel<T, false, false>);
  *kernel = reinterpret_cast<const void*>(k);
  return launch_dependent(k, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, int type,
                                const gp_fp8_matrix* q, const gp_fp8_matrix* qt, cudaStream_t stream,
                                const void** kernel, gp_plan* plan) {
  QuantArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  if (q) a.q = *q;
  if (qt) a.qt = *qt;
  const gp_fp8_matrix& any = q ? *q : *qt;
  a.e5m2 = any.format == GP_E5M2;
  a.fmax = a.e5m2 ? 57344.f : 448.f;
  a.tiles_c = (cols + kTile - 1) / kTile;
  const int64_t tiles = a.tiles_c * ((rows + kTile - 1) / kTile);
  plan->kernel = "fp8_quantize";
  plan->threads = kThreads;
  plan->bm = plan->bn = kTile;
  plan->tiles = tiles;
  plan->grid = static_cast<int32_t>(tiles);
  switch (type) {
    case GP_REAL_F16: return launch_type<__half>(a, any.group == kTile, tiles, stream, kernel);
    case GP_REAL_BF16: return launch_type<__nv_bfloat16>(a, any.group == kTile, tiles, stream, kernel);
    default: return launch_type<float>(a, any.group == kTile, tiles, stream, kernel);
  }
}

}  // namespace gp
