// Rows of bf16, f16 or f32 values as the operators around the indexer read
// and quantise them: eight values a lane, and the correctly rounded quotients
// that become e4m3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {

// Eight values as they lie in memory: one or two 16-byte pieces.
template <int TYPE>
struct Raw8 {
  uint4 v[TYPE == kRowF32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* src) {
#pragma unroll
    for (int i = 0; i < (TYPE == kRowF32 ? 2 : 1); ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (TYPE == kRowF32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x), x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z), x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (TYPE == kRowBf16)
          f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        else
          f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};

// The largest magnitude of values, from their bits: ordered like the numbers,
// infinities and NaN behind them, two 16-bit values or two f32 an instruction.
template <int TYPE>
struct Magnitude {
  static constexpr uint32_t kInf = TYPE == kRowF32 ? 0x7F800000u : TYPE == kRowBf16 ? 0x7F80u : 0x7C00u;
  uint32_t m = 0;
  __device__ __forceinline__ void add(const Raw8<TYPE>& x) {
    if constexpr (TYPE == kRowF32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m = __vimax3_u32(m, x.v[i].x & 0x7FFFFFFFu, x.v[i].y & 0x7FFFFFFFu);
        m = __vimax3_u32(m, x.v[i].z & 0x7FFFFFFFu, x.v[i].w & 0x7FFFFFFFu);
      }
    } else {
      m = __vimax3_u16x2(m, x.v[0].x & 0x7FFF7FFFu, x.v[0].y & 0x7FFF7FFFu);
      m = __vimax3_u16x2(m, x.v[0].z & 0x7FFF7FFFu, x.v[0].w & 0x7FFF7FFFu);
    }
  }
  __device__ __forceinline__ uint32_t top() const { return TYPE == kRowF32 ? m : max(m & 0xFFFFu, m >> 16); }
  // (of finite values)
  __device__ __forceinline__ float value() const {
    const uint32_t t = top();
    if constexpr (TYPE == kRowF32) return __uint_as_float(t);
    if constexpr (TYPE == kRowBf16) return __uint_as_float(t << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(t)));
  }
};

// The signs of eight values, where their codes have theirs.
template <int TYPE>
__device__ __forceinline__ uint2 code_signs(const Raw8<TYPE>& x) {
  uint2 s;
  if constexpr (TYPE == kRowF32) {
    s.x = __byte_perm(__byte_perm(x.v[0].x, x.v[0].y, 0x73), __byte_perm(x.v[0].z, x.v[0].w, 0x73), 0x5410);
    s.y = __byte_perm(__byte_perm(x.v[1].x, x.v[1].y, 0x73), __byte_perm(x.v[1].z, x.v[1].w, 0x73), 0x5410);
  } else {
    s.x = __byte_perm(x.v[0].x, x.v[0].y, 0x7531);
    s.y = __byte_perm(x.v[0].z, x.v[0].w, 0x7531);
  }
  return make_uint2(s.x & 0x80808080u, s.y & 0x80808080u);
}

// a / b for r = RN(1 / b) by Markstein's method (see paged_store.cu), divided
// where a step could underflow.
__device__ __forceinline__ float rounded_quotient(float a, float b, float r) {
  const float q = a * r;
  return a > 0x1p-80f && a < 0x1p120f ? fmaf(fmaf(-q, b, a), r, q) : __fdiv_rn(a, b);
}

// Whether quotients by `scale` have to be divided: a scale so small or large
// that a step of the method could leave the normal range, or with a
// significand of all ones.
__device__ __forceinline__ bool has_to_divide(float scale) {
  return !(scale > 0x1p-90f && scale < 0x1p90f) || (__float_as_uint(scale) & 0x7FFFFFu) == 0x7FFFFFu;
}

// The correctly rounded quotients x / scale of eight values (r = RN(1/scale),
// which has_to_divide does not hold for).  SIGNED: -0 / scale is -0, else 0; no
// other quotient lacks its value's sign.
template <bool SIGNED = true>
__device__ __forceinline__ void quotients8(const float (&x)[8], float scale, float r, float (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {  // two at a time
    const float2 v = make_float2(x[j], x[j + 1]), r2 = make_float2(r, r);
    const float2 q = __fmul2_rn(v, r2);
    const float2 e = __ffma2_rn(q, make_float2(-scale, -scale), v);
    const float2 z = __ffma2_rn(e, r2, q);
    y[j] = SIGNED ? copysignf(z.x, x[j]) : z.x;
    y[j + 1] = SIGNED ? copysignf(z.y, x[j + 1]) : z.y;
  }
}

// Eight e4m3 codes, saturating: max|x| / scale can round to just above 448.
__device__ __forceinline__ uint2 e4m3_codes8(const float (&y)[8]) {
  uint32_t codes[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
    codes[k] = lo | hi << 16;
  }
  return make_uint2(codes[0], codes[1]);
}

}  // namespace fp8idx
