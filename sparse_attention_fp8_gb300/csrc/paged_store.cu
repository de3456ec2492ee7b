// The quantising write into a paged cache (fp8_paged_store): each row of
// head_dim values becomes one f32 scale, max|x| / 448, and e4m3 codes of
// x / scale, and goes to its token's slot.
//
// D/16 lanes hold a row, eight values from each half a lane (16-byte loads of
// 16-bit types): the maximum is a butterfly among them, each lane stores its
// codes and the first one the scale.  The key and value rows of a token are
// neighbours in a page, so their lanes sit next to one another in a warp, which
// writes whole lines.  Codes follow the definition bit for bit: x / scale is
// the correctly rounded quotient, by Markstein's method (IBM J. Res. Dev. 34,
// 1990): with r the rounded reciprocal, q = x r and q + (x - q scale) r, each
// one fused operation, is the rounded quotient unless scale's significand is
// all ones; such rows, and scales so small or large that a step could leave
// the normal range, are divided.  (A division a value made the kernel bound by
// instructions: 32 us for 16384 tokens of 8 heads.)
// DRAM bound (2 or 4 bytes read and one written a value), so with many rows a
// lane loads its pieces of two rows before it works on them; with few the rows
// are spread over more warps.  16384 tokens of 8 heads, keys and values: 22.0 us,
// 4.6 TB/s of the 102 MB that have to move (68% of a copy's rate); 4096 index
// keys 1.9 us, 96 of them 1.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {
namespace {

constexpr int kStoreThreads = 128;  // (256: 23.8 us where this takes 22.0; the registers then hold fewer warps)

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

// a / b for r = RN(1 / b) (see above), divided where a step could underflow.
__device__ __forceinline__ float rounded_quotient(float a, float b, float r) {
  const float q = a * r;
  return a > 0x1p-80f && a < 0x1p120f ? fmaf(fmaf(-q, b, a), r, q) : __fdiv_rn(a, b);
}

}  // namespace

// PARTS 1: index cache (keys); 2: key/value cache.
template <int TYPE, int D, int PARTS, int kRows>
__global__ void __launch_bounds__(kStoreThreads) paged_store_kernel(const PagedStoreParams p) {
  constexpr int kLanes = D / 16, kPerWarp = 32 / kLanes;  // lanes of a row, rows a warp holds at a time
  constexpr int kItem = TYPE == kRowF32 ? 4 : 2;
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const uint32_t warp = blockIdx.x * (kStoreThreads / 32) + (threadIdx.x >> 5);
  const uint32_t per_token = static_cast<uint32_t>(p.heads) * PARTS;
  Raw8<TYPE> raw[kRows][2];  // values 8*sub .. and D/2 + 8*sub ..
  uint8_t* page[kRows];  // null: the row is not stored
  int32_t off[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    // rows are numbered token, head, part; a row's lanes agree on everything
    const uint32_t r = (warp * kRows + i) * kPerWarp + lane / kLanes;
    const uint32_t t = p.div_shift < 0 ? r : __umulhi(r, p.div_mul) >> p.div_shift, hp = r - t * per_token;
    const uint32_t h = hp / PARTS, part = hp % PARTS;
    page[i] = nullptr;
    off[i] = 0;
    if (t < p.tokens) {
      const int32_t slot = __ldg(p.slots + t);
      const uint8_t* src = static_cast<const uint8_t*>(p.x[part]) + t * p.token_stride[part] + h * p.head_stride[part] +
                           sub * 8 * kItem;
      raw[i][0].load(src);
      raw[i][1].load(src + D / 2 * kItem);
      if (slot >= 0 && slot < p.num_slots) {
        const int32_t block = slot >> p.block_shift;
        page[i] = p.cache + block * p.block_stride + h * p.cache_head_stride;
        off[i] = (slot - (block << p.block_shift)) * PARTS + static_cast<int32_t>(part);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float amax = 0.f;  // (a NaN does not count)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[8];
      raw[i][half].values(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (page[i] == nullptr) continue;  // (after the exchange: other rows' lanes take part in it)
    const float scale = rounded_quotient(amax, 448.f, 1.f / 448.f);
    const float r = __frcp_rn(scale);
    const bool divide = !(scale > 0x1p-90f && scale < 0x1p90f) || (__float_as_uint(scale) & 0x7FFFFFu) == 0x7FFFFFu;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[8], y[8];
      raw[i][half].values(x);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {  // two at a time
        const float2 v = make_float2(x[j], x[j + 1]), r2 = make_float2(r, r);
        const float2 q = __fmul2_rn(v, r2);
        const float2 e = __ffma2_rn(make_float2(-q.x, -q.y), make_float2(scale, scale), v);
        const float2 z = __ffma2_rn(e, r2, q);
        y[j] = copysignf(z.x, x[j]);  // (-0 / scale is -0)
        y[j + 1] = copysignf(z.y, x[j + 1]);
      }
      if (divide) {
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (amax is 0 for a row of zeros and NaN, too: the NaN stay)
          y[j] = amax != 0.f ? __fdiv_rn(x[j], scale) : x[j] == 0.f ? 0.f : x[j];
      }
      uint32_t codes[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // (saturating: max|x| / scale can round to just above 448)
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
        codes[k] = lo | hi << 16;
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(page[i] + off[i] * D + half * (D / 2) + sub * 8);
      // rows of the co-packed token cache (132 or 68 bytes) are only 4-byte aligned
      if (PARTS == 2 || p.block_shift > 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
      } else {
        dst[0] = codes[0];
        dst[1] = codes[1];
      }
    }
    if (sub == 0) reinterpret_cast<float*>(page[i] + (PARTS * D << p.block_shift))[off[i]] = scale;
  }
}

namespace {
using StoreKernel = void (*)(PagedStoreParams);
template <int TYPE, int ROWS>
StoreKernel store_instance(int head_dim, int parts) {
  if (head_dim == 128) return parts == 2 ? paged_store_kernel<TYPE, 128, 2, ROWS> : paged_store_kernel<TYPE, 128, 1, ROWS>;
  return parts == 2 ? paged_store_kernel<TYPE, 64, 2, ROWS> : paged_store_kernel<TYPE, 64, 1, ROWS>;
}
template <int ROWS>
StoreKernel store_instance(int row_type, int head_dim, int parts) {
  return row_type == kRowBf16  ? store_instance<kRowBf16, ROWS>(head_dim, parts)
         : row_type == kRowF16 ? store_instance<kRowF16, ROWS>(head_dim, parts)
                               : store_instance<kRowF32, ROWS>(head_dim, parts);
}
}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, int row_type, int head_dim, int sms, cudaStream_t stream) {
  const int parts = p.x[1] ? 2 : 1;
  // two rows a lane once that still makes eight CTAs for every SM
  const int64_t rows = p.tokens * p.heads * parts, per_cta = kStoreThreads / (head_dim / 16);
  const int per_lane = rows >= per_cta * 2 * 8 * sms ? 2 : 1;
  const StoreKernel kern = per_lane == 2 ? store_instance<2>(row_type, head_dim, parts)
                                         : store_instance<1>(row_type, head_dim, parts);
  kern<<<static_cast<unsigned>((rows + per_cta * per_lane - 1) / (per_cta * per_lane)), kStoreThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
