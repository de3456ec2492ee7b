// Attention over the selected positions of a paged key/value cache
// (fp8_paged_sparse_attn, fp8_mqa_sparse_attn_paged).
//
// One CTA per (row, key head, 32 query heads): tiles of 128 selected tokens
// are copied to shared memory, scores and the running maximum and sum of the
// softmax are f32, and the output stays in shared memory until the last tile.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {
namespace {

constexpr int kTile = 128;
constexpr int kHeadsPerCta = 32;
constexpr int kThreads = 256;

// The page row of entry `idx` of row `row`: the byte offset of the token's
// page and its place in the page, or false if the entry selects nothing.
__device__ __forceinline__ bool resolve(const SparseAttnParams& p, int row, int32_t idx, int64_t* block, int* off) {
  if (idx < 0) return false;
  int req = row / p.next_n;
  int64_t tok = idx;
  if (p.cu_seq_lens != nullptr) {
    int lo = 0, hi = p.n_req;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_seq_lens + mid) <= idx) lo = mid; else hi = mid;
    }
    if (__ldg(p.cu_seq_lens + lo) > idx || __ldg(p.cu_seq_lens + lo + 1) <= idx) return false;
    req = lo;
    tok = idx - __ldg(p.cu_seq_lens + lo);
  }
  const int64_t j = tok / p.block_size;
  if (j >= p.max_blocks) return false;
  const int32_t b = __ldg(p.block_tables + req * p.bt_stride + j);
  if (b < 0 || b >= p.num_blocks) return false;
  *block = b;
  *off = static_cast<int>(tok % p.block_size);
  return true;
}

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads) sparse_attn_kernel(const SparseAttnParams p) {
  extern __shared__ float attn_smem[];
  float* q_s = attn_smem;                          // [32][D]
  float* o_s = q_s + kHeadsPerCta * D;             // [32][D]
  float* s_s = o_s + kHeadsPerCta * D;             // [32][128]
  float* sc_s = s_s + kHeadsPerCta * kTile;        // [128][2]
  float* m_s = sc_s + 2 * kTile;                   // [32]
  float* l_s = m_s + kHeadsPerCta;                 // [32]
  float* f_s = l_s + kHeadsPerCta;                 // [32]
  uint8_t* kv_s = reinterpret_cast<uint8_t*>(f_s + kHeadsPerCta);  // [128][2*D + 4]
  constexpr int kPitch = 2 * D + 4;
  const int row = blockIdx.x, kvh = blockIdx.y, h0 = blockIdx.z * kHeadsPerCta;
  const int tid = threadIdx.x;
  const int nh = min(kHeadsPerCta, p.group - h0);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row / p.next_n * p.q_req_stride +
                           row % p.next_n * p.q_row_stride + (kvh * p.group + h0) * p.q_head_stride;
  for (int i = tid; i < nh * D; i += kThreads) {
    q_s[i] = __bfloat162float(q[i / D * p.q_head_stride + i % D]);
    o_s[i] = 0.f;
  }
  if (tid < nh) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  for (int t0 = 0; t0 < p.k; t0 += kTile) {
    __syncthreads();
    const int warp = tid >> 5, lane = tid & 31;
    for (int j = warp; j < kTile; j += kThreads / 32) {
      int64_t block = 0;
      int off = 0;
      const bool ok = t0 + j < p.k && resolve(p, row, __ldg(p.indices + row * p.idx_stride + t0 + j), &block, &off);
      const uint8_t* page = p.kv + block * p.block_stride + kvh * p.kv_head_stride;
      for (int w = lane; w < 2 * D / 4; w += 32)
        *reinterpret_cast<uint32_t*>(kv_s + j * kPitch + 4 * w) =
            ok ? __ldg(reinterpret_cast<const uint32_t*>(page + static_cast<int64_t>(off) * 2 * D) + w) : 0u;
      if (lane < 2) {
        const float* sc = reinterpret_cast<const float*>(page + static_cast<int64_t>(p.block_size) * 2 * D);
        sc_s[2 * j + lane] = ok ? __ldg(sc + 2 * off + lane) : (lane == 0 ? -1.f : 0.f);  // scale -1: not selected
      }
    }
    __syncthreads();
    for (int i = tid; i < nh * kTile; i += kThreads) {
      const int h = i / kTile, j = i % kTile;
      float a = 0.f;
      for (int d = 0; d < D; ++d) a += q_s[h * D + d] * e4m3(kv_s[j * kPitch + d]);
      s_s[i] = sc_s[2 * j] < 0.f ? -INFINITY : a * sc_s[2 * j] * p.scale_log2;
    }
    __syncthreads();
    for (int h = warp; h < nh; h += kThreads / 32) {
      float top = m_s[h];
      for (int j = lane; j < kTile; j += 32) top = fmaxf(top, s_s[h * kTile + j]);
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float sum = 0.f;
      for (int j = lane; j < kTile; j += 32) {
        const float e = top == -INFINITY ? 0.f : exp2f(s_s[h * kTile + j] - top);
        sum += e;
        s_s[h * kTile + j] = e * sc_s[2 * j + 1];
      }
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      __syncwarp();
      if (lane == 0) {
        const float f = m_s[h] == -INFINITY ? 0.f : exp2f(m_s[h] - top);
        f_s[h] = f;
        l_s[h] = l_s[h] * f + sum;
        m_s[h] = top;
      }
    }
    __syncthreads();
    for (int i = tid; i < nh * D; i += kThreads) {
      const int h = i / D, d = i % D;
      float a = o_s[i] * f_s[h];
      for (int j = 0; j < kTile; ++j) a += s_s[h * kTile + j] * e4m3(kv_s[j * kPitch + D + d]);
      o_s[i] = a;
    }
  }
  __syncthreads();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row / p.next_n * p.out_req_stride +
                       row % p.next_n * p.out_row_stride + (kvh * p.group + h0) * p.out_head_stride;
  for (int i = tid; i < nh * D; i += kThreads) {
    const float l = l_s[i / D];
    out[i / D * p.out_head_stride + i % D] = __float2bfloat16(l == 0.f ? 0.f : o_s[i] / l);
  }
  if (p.lse != nullptr && tid < nh)
    p.lse[static_cast<int64_t>(row) * p.heads + kvh * p.group + h0 + tid] =
        l_s[tid] == 0.f ? -INFINITY : (m_s[tid] + log2f(l_s[tid])) * 0.6931471805599453f;
}

cudaError_t launch_sparse_attn(const SparseAttnParams& p, int head_dim, int sms, int ctas_req, cudaStream_t stream) {
  (void)sms;
  (void)ctas_req;
  const auto kern = head_dim == 128 ? sparse_attn_kernel<128> : sparse_attn_kernel<64>;
  const int smem = 4 * (2 * kHeadsPerCta * head_dim + kHeadsPerCta * kTile + 2 * kTile + 3 * kHeadsPerCta) +
                   kTile * (2 * head_dim + 4);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.rows, p.kv_heads, (p.group + kHeadsPerCta - 1) / kHeadsPerCta);
  kern<<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
