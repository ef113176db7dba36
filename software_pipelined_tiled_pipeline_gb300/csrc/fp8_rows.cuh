// fp8_rows.cuh -- what the FP8 row kernels share: eight values at a time from
// and to memory, the scale of a group, and the 8-bit conversions.
#pragma once
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_internal.h"
#include "gp_device.cuh"

namespace gp {

// ---------------------------------------------------------------------------
// eight values of a row
// ---------------------------------------------------------------------------
template <typename T>
struct Raw8 {
  static constexpr int WORDS = static_cast<int>(sizeof(T)) * 8 / 16;
  uint4 w[WORDS];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// A thread's eight columns of a group of 128: with rows on 16-byte boundaries
// (vec) columns c .. c + 7, c a multiple of 8, else every 16th from (c / 8) mod
// 16 on, so that the 16 lanes of a group still read neighbouring values.  A
// group is the same 16 lanes either way.
struct Eight {
  int first, stride;
};
__device__ __forceinline__ Eight eight_columns(int c, bool vec) {
  return vec ? Eight{c, 1} : Eight{(c & ~127) + ((c >> 3) & 15), 16};
}

// The eight values of a row of `cols` (those past its end read as 0; cols 0: nothing is read).
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* row, int c, int cols, bool vec) {
  if (vec && c + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < Raw8<T>::WORDS; ++i) r.w[i] = reinterpret_cast<const uint4*>(row + c)[i];
    return;
  }
  const Eight e = eight_columns(c, vec);
  const T* p = row + e.first;
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    from_f32(0.f, t[i]);
    if (e.first + i * e.stride < cols) t[i] = p[i * e.stride];
  }
  memcpy(&r, t, sizeof(t));
}

// The values of one raw word: one FP32, or two 16-bit ones (the lower first).
template <typename T>
__device__ __forceinline__ float word_lo(uint32_t w) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(w << 16);
  __half2 h;
  memcpy(&h, &w, 4);
  return __low2float(h);
}
template <typename T>
__device__ __forceinline__ float word_hi(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(w & 0xFFFF0000u);
  __half2 h;
  memcpy(&h, &w, 4);
  return __high2float(h);
}
template <typename T>
__device__ __forceinline__ const uint32_t* words(const Raw8<T>& r) {
  return reinterpret_cast<const uint32_t*>(&r);
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4)
      v[i] = word_lo<T>(words(r)[i]);
    else
      v[i] = i & 1 ? word_hi<T>(words(r)[i / 2]) : word_lo<T>(words(r)[i / 2]);
  }
}

// Round eight FP32 values to T (nearest even).
template <typename T>
__device__ __forceinline__ void pack8(const float (&v)[8], Raw8<T>& r) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < Raw8<T>::WORDS * 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      memcpy(&w[i], &p, 4);
    } else {
      const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      memcpy(&w[i], &p, 4);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* row, const Raw8<T>& r, int c, int cols, bool vec) {
  if (vec && c + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < Raw8<T>::WORDS; ++i) reinterpret_cast<uint4*>(row + c)[i] = r.w[i];
    return;
  }
  const Eight e = eight_columns(c, vec);
  T* p = row + e.first;
  T t[8];
  memcpy(t, &r, sizeof(t));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e.first + i * e.stride < cols) p[i * e.stride] = t[i];
}

// The eight values of a vector of one of the gp_real types, as FP32.  aligned: the vector is on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8_as(float (&v)[8], const void* base, int c, int cols, bool vec, bool aligned) {
  Raw8<T> r;
  if (vec && !aligned) {     // columns c .. c + 7 one by one
    const T* p = static_cast<const T*>(base) + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f32(p[i]) : 0.f;
    return;
  }
  load8(r, static_cast<const T*>(base), c, cols, vec);
  unpack8(r, v);
}
__device__ __forceinline__ void load8_any(float (&v)[8], const void* base, int type, int c, int cols, bool vec,
                                          bool aligned) {
  if (type == GP_REAL_F32)
    load8_as<float>(v, base, c, cols, vec, aligned);
  else if (type == GP_REAL_BF16)
    load8_as<__nv_bfloat16>(v, base, c, cols, vec, aligned);
  else
    load8_as<__half>(v, base, c, cols, vec, aligned);
}

// Value k of eight as FP32.
template <typename T>
__device__ __forceinline__ float value_of(const Raw8<T>& r, int k) {
  if constexpr (sizeof(T) == 4) return word_lo<T>(words(r)[k]);
  return k & 1 ? word_hi<T>(words(r)[k / 2]) : word_lo<T>(words(r)[k / 2]);
}

// ---------------------------------------------------------------------------
// scales and 8-bit codes
// ---------------------------------------------------------------------------
// |x| as an ordered integer.  The bit patterns of non-negative floats order as
// the floats do and a NaN's lies above all of them, so an integer maximum of
// these also carries a NaN or an infinity of the group to its scale.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Magnitudes of raw values in their own bits: 16-bit types two to a word, with
// the same order and the same way of carrying a NaN.
template <typename T>
__device__ __forceinline__ uint32_t raw_abs(uint32_t word) {
  return word & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
}
template <typename T>
__device__ __forceinline__ uint32_t raw_max(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) return max(a, b);
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The magnitude in a word's only (32-bit types), lower or upper value, as FP32 bits.
template <typename T>
__device__ __forceinline__ uint32_t raw_to_bits(uint32_t word, int upper) {
  if constexpr (sizeof(T) == 4) return word;
  return __float_as_uint(upper ? word_hi<T>(word) : word_lo<T>(word));
}

constexpr float kScaleFloor = 5.42101086e-20f;   // 2^-64

// Scale of a group from its largest magnitude's bits, and the factor applied
// to its values.  Both are correctly rounded quotients.
struct GroupScale {
  float scale, inv;
};
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits, float fmax) {
  GroupScale g;
  g.scale = __fdiv_rn(__uint_as_float(amax_bits), fmax);
  if (g.scale < kScaleFloor) g.scale = kScaleFloor;   // false for NaN, which stays
  g.inv = __frcp_rn(g.scale);
  return g;
}

// Two values to two 8-bit codes (nearest even, saturated; NaN stays NaN), lo in the low byte.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  return fp8x2<E5M2>(a, b) | (fp8x2<E5M2>(c, d) << 16);
}

// The eight codes of a row (which begins on a 16-byte boundary).
__device__ __forceinline__ void store_codes8(uint8_t* row, uint2 codes, int c, int cols, bool vec) {
  if (vec && c + 8 <= cols) {
    *reinterpret_cast<uint2*>(row + c) = codes;
    return;
  }
  const Eight e = eight_columns(c, vec);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e.first + i * e.stride < cols)
      row[e.first + i * e.stride] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
}

}  // namespace gp
