// The quantising write into a paged cache whose blocks share one scale
// (fp8_paged_block_store): the new tokens of a block become e4m3 codes of
// x / scale, with one f32 scale for the keys and one for the values of a head.
//
// A run is a set of consecutive rows that go to consecutive slots of a block.
// Its scale is max|x| / 448 where the run opens the block; in a block that
// holds tokens already it is the old one, times the smallest power of two that
// reaches max|x| / 448: the codes written before then only lose one from their
// exponent for each doubling, which is exact but for the smallest ones, however
// often a block grows.
//
// A CTA takes the runs that start in its window of rows, one head's keys or
// values of each: the maximum in a first pass, the codes in a second one.
#include <cuda_runtime.h>

#include "rows.cuh"

namespace fp8idx {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// Four e4m3 codes times 2^-k (mul = 2^-k), rounded to nearest even.
__device__ __forceinline__ uint32_t shift_codes(uint32_t w, float mul) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 v = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3)));
    out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v.x * mul, v.y * mul), __NV_SATFINITE, __NV_E4M3))
           << (16 * i);
  }
  return out;
}

}  // namespace

template <int TYPE, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) block_store_kernel(const BlockStoreParams p) {
  constexpr int kItem = TYPE == kRowF32 ? 4 : 2, kLanes = D / 8, kRows = THREADS / kLanes, kWarps = THREADS / 32;
  __shared__ float warp_max[kWarps];
  __shared__ int32_t warp_run[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t at = blockIdx.x;
  const int part = at & 1u;
  at >>= 1;
  const uint32_t win = at / static_cast<uint32_t>(p.heads);
  const int h = static_cast<int>(at - win * p.heads);
  const int32_t t_end = min(static_cast<int32_t>(win + 1) * p.window, p.tokens);
  const uint8_t* const x = static_cast<const uint8_t*>(p.x[part]) + h * p.head_stride[part] + tid % kLanes * 8 * kItem;
  const int bs = 1 << p.block_shift;

#pragma unroll 1
  for (int32_t t0 = static_cast<int32_t>(win) * p.window; t0 < t_end; ++t0) {
    const int32_t slot = __ldg(p.slots + t0);
    if (slot < 0 || slot >= p.num_slots) continue;
    const int off0 = slot & (bs - 1);
    if (off0 != 0 && t0 > 0 && __ldg(p.slots + t0 - 1) == slot - 1) continue;  // inside a run
    // the run's rows: up to the first that goes elsewhere
    int run = bs - off0;
    {
      int mine = run;
#pragma unroll 1
      for (int j = 1 + tid; j < run; j += THREADS)
        if (t0 + j >= p.tokens || __ldg(p.slots + t0 + j) != slot + j) {
          mine = j;
          break;
        }
      mine = __reduce_min_sync(kFull, mine);
      if (kWarps > 1) {
        __syncthreads();  // (the last run's readers are done)
        if (lane == 0) warp_run[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mine = min(mine, warp_run[w]);
      }
      run = mine;
    }
    uint8_t* const page = p.cache + static_cast<int64_t>(slot >> p.block_shift) * p.block_stride + h * p.cache_head_stride;
    float* const scale_at = reinterpret_cast<float*>(page + (2 * D << p.block_shift)) + part;
    const float old = off0 ? *scale_at : 0.f;
    const uint8_t* const src = x + t0 * p.token_stride[part];

    // NaN and infinities do not count
    float amax = 0.f;
#pragma unroll 4
    for (int r = tid / kLanes; r < run; r += kRows) {
      Raw8<TYPE> raw;
      raw.load(src + r * p.token_stride[part]);
      float v[8];
      raw.values(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = fabsf(v[j]);
        amax = fmaxf(amax, a < INFINITY ? a : 0.f);
      }
    }
    amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
    if (kWarps > 1) {
      if (lane == 0) warp_max[warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, warp_max[w]);
    }
    const float need = rounded_quotient(amax, 448.f, 1.f / 448.f);
    float scale = need;
    int grow = 0;
    if (off0 != 0 && old != 0.f) {
      scale = old;
      if (need > old) {
        int en, eo;
        const float mn = frexpf(need, &en), mo = frexpf(old, &eo);
        grow = en - eo + (mn > mo ? 1 : 0);
        scale = ldexpf(old, grow);
      }
    }
    const float r1 = __frcp_rn(scale);
    const bool divide = has_to_divide(scale);
#pragma unroll 4
    for (int r = tid / kLanes; r < run; r += kRows) {
      Raw8<TYPE> raw;
      raw.load(src + r * p.token_stride[part]);
      float v[8], y[8];
      raw.values(v);
      quotients8(v, scale, r1, y);
      bool odd = divide;
#pragma unroll
      for (int j = 0; j < 8; ++j) odd |= !(fabsf(v[j]) < INFINITY);
      if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (NaN and infinities become NaN; scale 0: the others are zeros)
          y[j] = !(fabsf(v[j]) < INFINITY) ? NAN : scale != 0.f ? __fdiv_rn(v[j], scale) : 0.f;
      }
      *reinterpret_cast<uint2*>(page + (2 * (off0 + r) + part) * D + tid % kLanes * 8) = e4m3_codes8(y);
    }
    if (grow > 0) {  // the codes written before
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - min(grow, 100)) << 23);
#pragma unroll 1
      for (int r = tid / kLanes; r < off0; r += kRows) {
        uint2* const c = reinterpret_cast<uint2*>(page + (2 * r + part) * D + tid % kLanes * 8);
        const uint2 w = *c;
        *c = make_uint2(shift_codes(w.x, mul), shift_codes(w.y, mul));
      }
    }
    if (kWarps > 1) __syncthreads();  // every thread has read the old scale
    if (tid == 0) *scale_at = scale;
    t0 += run - 1;
  }
}

namespace {
using BlockStoreKernel = void (*)(BlockStoreParams);
template <int TYPE, int THREADS>
BlockStoreKernel block_store_instance(int head_dim) {
  return head_dim == 128 ? block_store_kernel<TYPE, 128, THREADS> : block_store_kernel<TYPE, 64, THREADS>;
}
template <int THREADS>
BlockStoreKernel block_store_instance(int row_type, int head_dim) {
  return row_type == kRowBf16  ? block_store_instance<kRowBf16, THREADS>(head_dim)
         : row_type == kRowF16 ? block_store_instance<kRowF16, THREADS>(head_dim)
                               : block_store_instance<kRowF32, THREADS>(head_dim);
}
}  // namespace

cudaError_t launch_block_store(BlockStoreParams& p, int row_type, int head_dim, int sms, cudaStream_t stream) {
  // A window of a block's rows has one or two runs of a prompt chunk; with few
  // rows, which may each be a run (decode), a window and a warp for every row.
  const int bs = 1 << p.block_shift;
  const int64_t per_row = 2ll * p.heads;
  const bool many = p.tokens / bs * per_row >= 4ll * sms;
  p.window = many ? bs : 1;
  const int64_t ctas = (p.tokens + p.window - 1) / p.window * per_row;
  if (many)
    block_store_instance<128>(row_type, head_dim)<<<static_cast<unsigned>(ctas), 128, 0, stream>>>(p);
  else
    block_store_instance<32>(row_type, head_dim)<<<static_cast<unsigned>(ctas), 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
