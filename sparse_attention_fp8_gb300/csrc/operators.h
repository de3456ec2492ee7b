// Parameter blocks and launchers of the operators around the indexer: the
// step tables, the quantising paged store and the sparse attention.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace fp8idx {

// ------------------------------------------------------------ step tables
constexpr int kStepThreads = 1024;
struct StepTablesParams {
  const int32_t* old_lens;
  const int32_t* new_lens;
  const int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* cu_new;
  int32_t* slots;
  int32_t* counts;
  int32_t* cu_seq;  // or null
  int32_t* ks;      // or null
  int32_t* ke;      // or null
  int64_t bt_stride;
  int64_t rows;
  int64_t free_cap;
  int32_t batch;
  int32_t max_blocks;
  int32_t block_size;
};
// three prefix sums of batch + 1 entries
__host__ __device__ constexpr int step_smem_bytes(int batch) { return 3 * 4 * (batch + 1); }
cudaError_t launch_step_tables(const StepTablesParams& p, int grid, cudaStream_t stream);

// ------------------------------------------------------------ paged store
enum RowType : int { kRowBf16 = 0, kRowF16 = 1, kRowF32 = 2 };
struct PagedStoreParams {
  const void* x[2];            // keys, values (or null)
  int64_t token_stride[2];     // bytes
  int64_t head_stride[2];      // bytes
  const int32_t* slots;
  uint8_t* cache;
  int64_t block_stride;        // bytes between blocks
  int64_t cache_head_stride;   // bytes between heads
  int64_t num_slots;           // num_blocks * block_size
  int64_t tokens;
  int32_t heads;
  int32_t block_size;
};
cudaError_t launch_paged_store(const PagedStoreParams& p, int row_type, int head_dim, cudaStream_t stream);

// ------------------------------------------------------- sparse attention
struct SparseAttnParams {
  const void* q;
  void* out;
  float* lse;                   // [rows][heads] or null
  const uint8_t* kv;
  const int32_t* indices;
  const int32_t* block_tables;
  const int32_t* cu_seq_lens;   // prefill: [n_req + 1]; decode: null
  int64_t q_req_stride, q_row_stride, q_head_stride;        // elements; row r is (r / next_n, r % next_n)
  int64_t out_req_stride, out_row_stride, out_head_stride;
  int64_t idx_stride;
  int64_t bt_stride;
  int64_t block_stride, kv_head_stride;                     // bytes
  int64_t num_blocks;
  int32_t rows, heads, kv_heads, group;                     // group: query heads per key head
  int32_t next_n;                                           // prefill: 1
  int32_t k, max_blocks, block_size, n_req;
  float scale_log2;                                         // softmax_scale * log2(e)
};
constexpr int kAttnMaxK = 2048;
constexpr int kAttnMaxGroup = 128;
cudaError_t launch_sparse_attn(const SparseAttnParams& p, int head_dim, int sms, int ctas_req, cudaStream_t stream);

}  // namespace fp8idx
