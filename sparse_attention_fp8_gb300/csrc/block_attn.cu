// Dense attention over a paged e4m3 cache whose blocks share one scale
// (fp8_paged_block_attn).
//
// A warp takes one query row and head; its lanes hold the channels and walk
// the row's positions one after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

template <int D>
__global__ void __launch_bounds__(128) block_attn_kernel(const BlockAttnParams p) {
  constexpr int kPer = D / 32;  // channels of a lane
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t row = unit / p.heads;
  const int h = static_cast<int>(unit - row * p.heads);
  if (row >= p.rows || row >= __ldg(p.cu_new + p.n_req)) return;
  int a = 0, b = p.n_req;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (__ldg(p.cu_new + mid) <= row) a = mid; else b = mid;
  }
  const int32_t ctx = __ldg(p.context_lens + a);
  const int64_t pos = static_cast<int64_t>(ctx) - __ldg(p.cu_new + a + 1) + row;
  const int64_t hi = min(min(pos + 1, static_cast<int64_t>(ctx)), static_cast<int64_t>(p.max_blocks) << p.block_shift);
  const int64_t lo = p.window > 0 ? max(pos - p.window + 1, static_cast<int64_t>(0)) : 0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * p.q_row_stride + h * p.q_head_stride;
  float qv[kPer], o[kPer] = {};
  for (int i = 0; i < kPer; ++i) qv[i] = __bfloat162float(q[lane * kPer + i]);
  float m = -3e38f, l = 0.f;
  const int bs = 1 << p.block_shift;
  for (int64_t at = lo; at < hi; ++at) {
    const int32_t block = __ldg(p.block_tables + a * p.bt_stride + (at >> p.block_shift));
    if (block < 0 || block >= p.num_blocks) continue;
    const uint8_t* page = p.kv + block * p.block_stride + h / p.group * p.head_stride;
    const float2 scales = *reinterpret_cast<const float2*>(page + 2 * D * bs);
    const uint8_t* kr = page + (at & (bs - 1)) * 2 * D;
    float s = 0.f, v[kPer];
    for (int i = 0; i < kPer; ++i) {
      s += qv[i] * __half2float(__half(__nv_cvt_fp8_to_halfraw(kr[lane * kPer + i], __NV_E4M3)));
      v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(kr[D + lane * kPer + i], __NV_E4M3)));
    }
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    s *= scales.x * p.scale_log2;
    const float top = fmaxf(m, s), f = exp2f(m - top), e = exp2f(s - top);
    l = l * f + e;
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + e * scales.y * v[i];
    m = top;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_row_stride + h * p.out_head_stride;
  for (int i = 0; i < kPer; ++i) out[lane * kPer + i] = __float2bfloat16(l == 0.f ? 0.f : o[i] / l);
  if (p.lse && lane == 0) p.lse[row * p.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_block_attn(const BlockAttnParams& p, int head_dim, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.rows) * p.heads;
  (head_dim == 128 ? block_attn_kernel<128> : block_attn_kernel<64>)
      <<<static_cast<unsigned>((units + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
