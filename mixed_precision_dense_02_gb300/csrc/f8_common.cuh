// What the kernels that make 8-bit operands share: element access by type,
// the scale of a block and the rounding to 8 bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"

namespace mmagb {

constexpr int kScaleBlock = 128;

// A 16-byte vector of T as floats.  kN elements per vector.
template <class T>
struct Vec;

template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ static void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                      __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static float round(float v) { return v; }
};

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};

template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  __device__ static void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static __half round(float v) { return __float2half_rn(v); }
};

// Clear what lies past a row's n elements in its vector v.
template <class T>
__device__ __forceinline__ void clear_tail(int64_t v, int64_t n,
                                           float (&f)[Vec<T>::kN]) {
  constexpr int E = Vec<T>::kN;
  if ((v + 1) * E > n) {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (v * E + j >= n) f[j] = 0.f;
  }
}

// The 16 bytes of a row's vector `v`, zeros beyond the row.  The last vector
// of a row may reach past its n elements (TAIL: they are not a multiple of
// a vector's), but never past the 16-byte chunk that holds its last one,
// because rows start on 16-byte boundaries; clear_tail clears what lies there.
template <class T>
__device__ __forceinline__ uint4 load_raw(const T* row, int64_t v, int64_t n) {
  return v * Vec<T>::kN < n ? __ldg(reinterpret_cast<const uint4*>(row) + v)
                            : make_uint4(0, 0, 0, 0);
}

template <class T, bool TAIL = true>
__device__ __forceinline__ void load_row(const T* row, int64_t v, int64_t n,
                                         float (&f)[Vec<T>::kN]) {
  Vec<T>::unpack(load_raw(row, v, n), f);
  if constexpr (TAIL) clear_tail<T>(v, n, f);
}

// (v is a vector of the row)
template <class T, bool TAIL = true>
__device__ __forceinline__ void store_row(T* row, int64_t v, int64_t n,
                                          const float (&f)[Vec<T>::kN]) {
  constexpr int E = Vec<T>::kN;
  if (!TAIL || (v + 1) * E <= n) {
    *(reinterpret_cast<uint4*>(row) + v) = Vec<T>::pack(f);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (v * E + j < n) row[v * E + j] = Vec<T>::round(f[j]);
  }
}

// Largest magnitude as the bits of |x|: integer order is the order of the
// magnitudes, with NaN above infinity, so a NaN among them wins.
__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __float_as_uint(x) & 0x7FFFFFFFu;
}

// The larger of two magnitudes, NaN if one is.
__device__ __forceinline__ float abs_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// The largest of three.
__device__ __forceinline__ float abs_max(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool E5M2>
constexpr float f8_max() { return E5M2 ? 57344.f : 448.f; }

// m over the format's largest value (7 times a power of two), rounded to
// nearest: with a reciprocal of two terms, r - hi < 2^-22 r and lo the rest to
// 24 bits, the sum is 2^-45 off, and no quotient by 7 is nearer than 1/14 of
// its last place to the middle between two numbers.  Small m are multiplied by
// 2^64, so that m lo is a normal number.
template <bool E5M2>
__device__ __forceinline__ float over_f8_max(float m) {
  constexpr double r = 1.0 / (E5M2 ? 57344.0 : 448.0);
  constexpr float hi = float(r * (1.0 - 0x1p-23)), lo = float(r - double(hi));
  static_assert(lo > 0.f);
  const bool small = m < 0x1p-64f;
  const float x = small ? m * 0x1p64f : m;
  const float s = fmaf(x, hi, x * lo);
  return small ? s * 0x1p-64f : s;
}

// The scale of a block whose largest magnitude is `m`: that over the format's
// largest value, at least 2^-126 (so that a block of zeros, or of values whose
// quotient underflows, has a scale that can be divided by).  With pow2 it is
// rounded up to a power of two.  A NaN or infinity in the block makes the scale
// one.
template <bool E5M2>
__device__ __forceinline__ float block_scale(float m, bool pow2) {
  float s = over_f8_max<E5M2>(m);
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  if (pow2) {
    uint32_t b = __float_as_uint(s);
    if ((b & 0x7FFFFFu) && b < 0x7F800000u) b = (b + 0x800000u) & 0xFF800000u;
    s = __uint_as_float(b);
  }
  return s;
}

// Division by a block's scale s.  x times 1 / s rounds twice, and x / s often
// lies half-way between two 8-bit values, where the second rounding decides.
// So the reciprocal has two terms, hi a little below 1 / s and lo = hi (1 - hi
// s), short of 1 / s - hi by 2^-42 of it, and x / s is fma(x, hi, x lo): an
// exact tie stays one, and any other quotient is that of FP32 but for the last
// place of one in some 10^6 (s above 2^100, where lo is subnormal: one in some
// 10^4).  lo > 0, so that zeros keep their sign.  s infinite: finite x give 0,
// infinite ones NaN.
struct Divisor {
  float hi, lo;
  Divisor() = default;
  __device__ __forceinline__ explicit Divisor(float s) {
    float r;  // within 2^-23 of 1 / s
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    hi = r * (1.f - 0x1p-22f);
    lo = s < INFINITY ? fmaf(-hi, s, 1.f) * hi : 0.f;
  }
  // that of another lane of the warp
  __device__ __forceinline__ Divisor from(int lane) const {
    Divisor d;
    d.hi = __shfl_sync(0xffffffffu, hi, lane);
    d.lo = __shfl_sync(0xffffffffu, lo, lane);
    return d;
  }
  __device__ __forceinline__ float2 operator()(float a, float b) const {
    const float2 x = make_float2(a, b);
    return __ffma2_rn(x, make_float2(hi, hi), __fmul2_rn(x, make_float2(lo, lo)));
  }
};

// Two values, already divided by their scale, in 8 bits (to nearest, ties
// to even; beyond the largest value that value; NaN stays NaN).
template <bool E5M2>
__device__ __forceinline__ uint32_t to_f8x2(float2 v) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE,
                                           E5M2 ? __NV_E5M2 : __NV_E4M3));
}

// Store E values of vector v of a row in 8 bits, over their scale.
template <bool E5M2, int E, bool TAIL = true>
__device__ __forceinline__ void store_f8(uint8_t* row, int64_t v, int64_t n,
                                         const float (&y)[E], const Divisor& d) {
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i)
    w[i] = to_f8x2<E5M2>(d(y[4 * i], y[4 * i + 1])) |
           (to_f8x2<E5M2>(d(y[4 * i + 2], y[4 * i + 3])) << 16);
  if (!TAIL || (v + 1) * E <= n) {
    if constexpr (E == 8)
      *reinterpret_cast<uint2*>(row + v * 8) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(row + v * 4) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (v * E + j < n) row[v * E + j] = uint8_t(w[j / 4] >> (8 * (j & 3)));
  }
}

}  // namespace mmagb
