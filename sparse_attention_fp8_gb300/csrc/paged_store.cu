// The quantising write into a paged cache (fp8_paged_store): each row of
// head_dim values becomes one f32 scale, max|x| / 448, and e4m3 codes of
// x / scale, and goes to its token's slot.
//
// D/8 lanes hold a row, eight values each (16-byte loads of 16-bit types):
// the maximum is a butterfly among them, each lane stores its eight codes and
// the first one the scale.  The key and value rows of a token are neighbours
// in a page, so their lanes sit next to one another in a warp, which then
// writes whole lines.  The division is IEEE (codes follow the definition bit
// for bit).  DRAM bound: 2 or 4 bytes read and one written a value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {
namespace {

constexpr int kStoreThreads = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t* src, float (&x)[8]) {
  if constexpr (TYPE == kRowF32) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(src)), b = __ldcs(reinterpret_cast<const float4*>(src) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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

}  // namespace

// PARTS 1: index cache (keys); 2: key/value cache.
template <int TYPE, int D, int PARTS>
__global__ void __launch_bounds__(kStoreThreads) paged_store_kernel(const PagedStoreParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kItem = TYPE == kRowF32 ? 4 : 2;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x;
  const int sub = static_cast<int>(idx % kLanes);
  const int part = static_cast<int>((idx / kLanes) % PARTS);
  const int64_t th = idx / (kLanes * PARTS);
  const int64_t t = th / p.heads;
  const int h = static_cast<int>(th - t * p.heads);
  if (t >= p.tokens) return;
  const int32_t slot = __ldg(p.slots + t);
  if (slot < 0 || slot >= p.num_slots) return;  // the whole row's lanes leave together
  float x[8];
  load8<TYPE>(static_cast<const uint8_t*>(p.x[part]) + t * p.token_stride[part] + h * p.head_stride[part] +
                  sub * 8 * kItem, x);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const uint32_t row_mask = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(row_mask, amax, d));
  const float scale = __fdiv_rn(amax, 448.f);
  uint32_t codes[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (saturating: max|x| / scale can round to just above 448)
      const float y = amax == 0.f ? 0.f : __fdiv_rn(x[4 * i + j], scale);
      c |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3)) << (8 * j);
    }
    codes[i] = c;
  }
  const int64_t block = slot / p.block_size, off = slot % p.block_size;
  uint8_t* page = p.cache + block * p.block_stride + h * p.cache_head_stride;
  // rows of the co-packed token cache (132 or 68 bytes) are only 4-byte aligned
  uint32_t* dst = reinterpret_cast<uint32_t*>(page + (off * PARTS + part) * D + sub * 8);
  if (PARTS == 2 || p.block_size > 1) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
  } else {
    dst[0] = codes[0];
    dst[1] = codes[1];
  }
  if (sub == 0)
    reinterpret_cast<float*>(page + static_cast<int64_t>(p.block_size) * PARTS * D)[off * PARTS + part] = scale;
}

namespace {
template <int TYPE>
void (*store_instance(int head_dim, int parts))(PagedStoreParams) {
  if (head_dim == 128) return parts == 2 ? paged_store_kernel<TYPE, 128, 2> : paged_store_kernel<TYPE, 128, 1>;
  return parts == 2 ? paged_store_kernel<TYPE, 64, 2> : paged_store_kernel<TYPE, 64, 1>;
}
}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, int row_type, int head_dim, cudaStream_t stream) {
  const int parts = p.x[1] ? 2 : 1;
  auto kern = row_type == kRowBf16  ? store_instance<kRowBf16>(head_dim, parts)
              : row_type == kRowF16 ? store_instance<kRowF16>(head_dim, parts)
                                    : store_instance<kRowF32>(head_dim, parts);
  const int64_t lanes = p.tokens * p.heads * parts * (head_dim / 8);
  kern<<<static_cast<unsigned>((lanes + kStoreThreads - 1) / kStoreThreads), kStoreThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
