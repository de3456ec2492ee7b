// Block tables, slots and windows of a serving step from request lengths
// (fp8idx_paged_step_tables).
//
// Three prefix sums over the requests -- new tokens, context lengths, blocks
// newly needed -- turn every output into an independent element: row t and
// the f-th new block each find their request by a binary search.  Every CTA
// computes the sums itself (at most 4096 requests: four a thread, in 64 bits
// so that nothing wraps) and then takes its share of the rows and blocks, so
// one launch does the step and no CTA waits for another: a row whose block is
// dealt in this step takes it from the free list, not from the table that
// another CTA is writing.  The free list is read and its new length goes to
// counts[2], which keeps the call repeatable and its CTAs free of races.
// Latency bound (20 bytes a request, at most 16 a row, 8 a block dealt): lengths,
// three block-wide sums, searches, table.  64 decode requests 4.8 us, 8192 new
// tokens 5.4 us, 4096 requests with blocks of one token 8.6 us.
#include <cuda_runtime.h>

#include "operators.h"

namespace fp8idx {
namespace {

constexpr int32_t kIntMax = 0x7FFFFFFF;
__device__ __forceinline__ int32_t saturate(int64_t v) { return v > kIntMax ? kIntMax : static_cast<int32_t>(v); }

// Largest i in [0, n) with a[i] <= v (a ascending, a[0] <= v).
__device__ __forceinline__ int find(const int32_t* a, int n, int32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(kStepThreads, 1) step_tables_kernel(const StepTablesParams p) {
  extern __shared__ int32_t step_smem[];
  const int B = p.batch;
  int32_t* cu_new = step_smem;             // [B + 1]
  int32_t* cu_seq = cu_new + B + 1;        // [B + 1]
  int32_t* cu_blk = cu_seq + B + 1;        // [B + 1]: new blocks
  __shared__ int64_t warp_sum[3][kStepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t bs = p.block_size;
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * bs;

  constexpr int kPer = kMaxBatch / kStepThreads;
  int64_t mine[3] = {0, 0, 0};
  int64_t part[3][kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
#pragma unroll
    for (int s = 0; s < 3; ++s) part[s][i] = mine[s];
    if (b < B) {
      const int64_t o = max(__ldg(p.old_lens + b), 0), n = max(__ldg(p.new_lens + b), 0);
      const int64_t c = min(o + n, cap);
      mine[0] += n;
      mine[1] += c;
      mine[2] += max((c + bs - 1) / bs - (o + bs - 1) / bs, static_cast<int64_t>(0));
    }
  }
  int64_t before[3];
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    int64_t v = mine[s];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (lane == 31) warp_sum[s][warp] = v;
    before[s] = v - mine[s];
  }
  __syncthreads();
  if (warp < 3) {
    int64_t v = warp_sum[warp][lane];
    const int64_t own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    __syncwarp();
    warp_sum[warp][lane] = v - own;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    if (b <= B) {
      cu_new[b] = saturate(warp_sum[0][warp] + before[0] + part[0][i]);
      cu_seq[b] = saturate(warp_sum[1][warp] + before[1] + part[1][i]);
      cu_blk[b] = saturate(warp_sum[2][warp] + before[2] + part[2][i]);
    }
  }
  if (B == kMaxBatch && tid == kStepThreads - 1) {  // the totals, one past the last thread's requests
    cu_new[B] = saturate(warp_sum[0][warp] + before[0] + mine[0]);
    cu_seq[B] = saturate(warp_sum[1][warp] + before[1] + mine[1]);
    cu_blk[B] = saturate(warp_sum[2][warp] + before[2] + mine[2]);
  }
  __syncthreads();

  const int32_t count = static_cast<int32_t>(
      min(static_cast<int64_t>(max(__ldg(p.free_count), 0)), p.free_cap));
  const int32_t wanted = cu_blk[B], total = cu_new[B];
  if (blockIdx.x == 0) {
    for (int b = tid; b <= B; b += kStepThreads) {
      p.cu_new[b] = cu_new[b];
      if (p.cu_seq) p.cu_seq[b] = cu_seq[b];
      if (b < B)
        p.context_lens[b] = static_cast<int32_t>(min(static_cast<int64_t>(max(__ldg(p.old_lens + b), 0)) +
                                                         max(__ldg(p.new_lens + b), 0), cap));
    }
    if (tid == 0) {
      const int32_t dealt = min(wanted, count);
      p.counts[0] = total;
      p.counts[1] = dealt;
      p.counts[2] = count - dealt;
      p.counts[3] = wanted - dealt;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kStepThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kStepThreads + tid;
  for (int64_t f = first; f < wanted; f += step) {
    const int b = find(cu_blk, B, static_cast<int32_t>(f));
    const int64_t held = (static_cast<int64_t>(max(__ldg(p.old_lens + b), 0)) + bs - 1) / bs;
    p.block_tables[b * p.bt_stride + held + (f - cu_blk[b])] = f < count ? __ldg(p.free_blocks + (count - 1 - f)) : -1;
  }
  for (int64_t t = first; t < p.rows; t += step) {
    int32_t slot = -1, lo = 0, hi = 0;
    if (t < total) {
      const int b = find(cu_new, B, static_cast<int32_t>(t));
      const int64_t o = max(__ldg(p.old_lens + b), 0), n = max(__ldg(p.new_lens + b), 0);
      const int64_t pos = o + (t - cu_new[b]);
      const int64_t j = pos / bs, held = (o + bs - 1) / bs;
      lo = cu_seq[b];
      hi = saturate(static_cast<int64_t>(lo) + min(pos + 1, min(o + n, cap)));
      if (j < p.max_blocks) {
        int32_t block;
        if (j < held) {
          block = p.block_tables[b * p.bt_stride + j];
        } else {
          const int64_t f = cu_blk[b] + (j - held);
          block = f < count ? __ldg(p.free_blocks + (count - 1 - f)) : -1;
        }
        const int64_t s = static_cast<int64_t>(block) * bs + pos % bs;
        if (block >= 0 && s <= kIntMax) slot = static_cast<int32_t>(s);
      }
    }
    p.slots[t] = slot;
    if (p.ks) p.ks[t] = lo;
    if (p.ke) p.ke[t] = hi;
  }
}

cudaError_t launch_step_tables(const StepTablesParams& p, int grid, cudaStream_t stream) {
  const int smem = step_smem_bytes(p.batch);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(step_tables_kernel), smem);
  if (e != cudaSuccess) return e;
  step_tables_kernel<<<grid, kStepThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
