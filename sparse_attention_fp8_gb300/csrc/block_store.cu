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
// values of each, a run at a time: its rows stay in the registers (eight 8-value
// pieces a thread at most) between the maximum and the codes.  Where runs start
// and end shows in two masks of the window's rows and a block's after it, made
// by all threads at once.  Maxima are taken of the values' bits, two 16-bit
// values an instruction, and tell NaN and infinities, too.
//
// Read once and written once.  12288 bf16 rows of 8 heads of 128 in blocks of 64
// take 17.1 us, 4.4 TB/s: the chain slots - rows - maximum - codes of a CTA, with
// eight CTAs of 64 registers on an SM (loads are what most warps wait for), and
// the arithmetic (with floating-point maxima and signs value by value, 92
// registers, 19.2 us).  Fewer registers for f32 rows (4.4 us instead of 4.1 for
// 3 heads of 64) and rows fetched into L2 before their slots are known (17.3) do
// not pay.  The same
// rows in f32 take 21.8 us, 5.8 TB/s; a decode step of 96 rows 3.5 us, a launch.
#include <cuda_runtime.h>

#include <algorithm>

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

// THREADS: an eighth of the pieces of a block's rows.
template <int TYPE, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) block_store_kernel(const BlockStoreParams p) {
  constexpr int kItem = TYPE == kRowF32 ? 4 : 2, kLanes = D / 8, kRows = THREADS / kLanes, kWarps = THREADS / 32, kHeld = 8;
  constexpr int kMasks = 2 * 128 / 32;
  __shared__ float warp_max[kWarps];
  __shared__ uint32_t goes_on[kMasks], starts[kMasks];  // row i continues a run; starts one (in the window)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t at = blockIdx.x;
  const int part = at & 1u;
  at >>= 1;
  const uint32_t win = at / static_cast<uint32_t>(p.heads);
  const int h = static_cast<int>(at - win * p.heads);
  const int32_t t_base = static_cast<int32_t>(win) * p.window;
  const int bs = 1 << p.block_shift, n = p.window + bs;
#pragma unroll 1
  for (int i = tid; i < (n + 31 & ~31); i += THREADS) {
    const int64_t t = static_cast<int64_t>(t_base) + i;
    bool on = false, first = false;
    if (i < n && t < p.tokens) {
      const int32_t slot = __ldg(p.slots + t), before = t > 0 ? __ldg(p.slots + t - 1) : -1;
      const bool valid = slot >= 0 && slot < p.num_slots;
      on = valid && (slot & (bs - 1)) != 0 && before == slot - 1 && t > 0;
      first = valid && !on && i < p.window;
    }
    const uint32_t a = __ballot_sync(kFull, on), b = __ballot_sync(kFull, first);
    if (lane == 0) {
      goes_on[i >> 5] = a;
      starts[i >> 5] = b;
    }
  }
  if (kWarps > 1) __syncthreads(); else __syncwarp();
  const uint8_t* const x = static_cast<const uint8_t*>(p.x[part]) + h * p.head_stride[part] + tid % kLanes * 8 * kItem;
  const int row = tid / kLanes;

#pragma unroll 1
  for (int word = 0; word * 32 < p.window; ++word) {
#pragma unroll 1
    for (uint32_t left = starts[word]; left != 0u; left &= left - 1u) {
      const int i0 = word * 32 + __ffs(left) - 1;
      int end = i0 + 1;
      while (end < n) {  // the first row that does not go on
        const uint32_t stop = ~goes_on[end >> 5] >> (end & 31);
        if (stop != 0u) {
          end += __ffs(stop) - 1;
          break;
        }
        end = (end | 31) + 1;
      }
      const int32_t t0 = t_base + i0;
      const int run = min(end, n) - i0;
      // (read again: if someone writes it meanwhile, the block and its rows stay in range)
      const int32_t slot = min(max(__ldg(p.slots + t0), 0), p.num_slots - 1);
      const int off0 = slot & (bs - 1);
      uint8_t* const page = p.cache + static_cast<int64_t>(slot >> p.block_shift) * p.block_stride + h * p.cache_head_stride;
      float* const scale_at = reinterpret_cast<float*>(page + (2 * D << p.block_shift)) + part;
      const uint8_t* const src = x + t0 * p.token_stride[part];
      Raw8<TYPE> raw[kHeld] = {};
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (row + k * kRows < run) raw[k].load(src + (row + k * kRows) * p.token_stride[part]);
      const float old = off0 ? *scale_at : 0.f;

      Magnitude<TYPE> mag;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) mag.add(raw[k]);
      const bool odd = mag.top() >= Magnitude<TYPE>::kInf;
      float amax = mag.value();
      if (__any_sync(kFull, odd)) {  // NaN and infinities do not count
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          float v[8];
          raw[k].values(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]) < INFINITY ? fabsf(v[j]) : 0.f);
        }
      }
      amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
      if (kWarps > 1) {
        if (lane == 0) warp_max[warp] = amax;
        __syncthreads();  // (and every thread has read the old scale)
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
      const bool divide = odd || has_to_divide(scale);
      uint8_t* const dst = page + (2 * off0 + part) * D + tid % kLanes * 8;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int r = row + k * kRows;
        if (r >= run || off0 + r >= bs) break;
        float v[8], y[8];
        raw[k].values(v);
        uint2 sign = make_uint2(0u, 0u);
        if (!divide) {
          quotients8<false>(v, scale, r1, y);
          sign = code_signs<TYPE>(raw[k]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)  // (NaN and infinities become NaN; scale 0: the others are zeros)
            y[j] = !(fabsf(v[j]) < INFINITY) ? NAN : scale != 0.f ? __fdiv_rn(v[j], scale) : 0.f;
        }
        const uint2 codes = e4m3_codes8(y);
        *reinterpret_cast<uint2*>(dst + r * 2 * D) = make_uint2(codes.x | sign.x, codes.y | sign.y);
      }
      if (grow > 0) {  // the codes written before
        const float mul = __uint_as_float(static_cast<uint32_t>(127 - min(grow, 100)) << 23);
#pragma unroll 1
        for (int r = row; r < off0; r += kRows) {
          uint2* const c = reinterpret_cast<uint2*>(page + (2 * r + part) * D + tid % kLanes * 8);
          const uint2 w = *c;
          *c = make_uint2(shift_codes(w.x, mul), shift_codes(w.y, mul));
        }
      }
      if (kWarps == 1) __syncwarp();
      if (tid == 0) *scale_at = scale;
      if (kWarps > 1) __syncthreads();  // warp_max is free again
    }
  }
}

namespace {
using BlockStoreKernel = void (*)(BlockStoreParams);
template <int TYPE, int D>
BlockStoreKernel block_store_instance(int threads) {
  if constexpr (D == 128)
    return threads == 32    ? block_store_kernel<TYPE, D, 32>
           : threads == 64  ? block_store_kernel<TYPE, D, 64>
           : threads == 128 ? block_store_kernel<TYPE, D, 128> : block_store_kernel<TYPE, D, 256>;
  else
    return threads == 32 ? block_store_kernel<TYPE, D, 32>
           : threads == 64 ? block_store_kernel<TYPE, D, 64> : block_store_kernel<TYPE, D, 128>;
}
template <int D>
BlockStoreKernel block_store_instance(int row_type, int threads) {
  return row_type == kRowBf16  ? block_store_instance<kRowBf16, D>(threads)
         : row_type == kRowF16 ? block_store_instance<kRowF16, D>(threads) : block_store_instance<kRowF32, D>(threads);
}
}  // namespace

cudaError_t launch_block_store(BlockStoreParams& p, int row_type, int head_dim, int sms, cudaStream_t stream) {
  // Windows of a block's rows, which have one or two runs of a prompt chunk, once
  // they make 8 CTAs for every SM; with fewer rows, which may each be a run
  // (decode), smaller ones.  (At 16, 32 and 64 CTAs the 12288 rows take the same,
  // the same and 9% more, 96 rows of 16 requests 4.4 us instead of 3.6.)
  const int bs = 1 << p.block_shift, threads = std::max(bs * (head_dim / 8) / 8, 32);
  const int64_t per_row = 2ll * p.heads;
  p.window = 1;
  while (p.window < bs && p.tokens / p.window * per_row > 8ll * sms) p.window *= 2;
  const int64_t ctas = (p.tokens + p.window - 1ll) / p.window * per_row;
  const BlockStoreKernel kern = head_dim == 128 ? block_store_instance<128>(row_type, threads)
                                                : block_store_instance<64>(row_type, threads);
  kern<<<static_cast<unsigned>(ctas), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
