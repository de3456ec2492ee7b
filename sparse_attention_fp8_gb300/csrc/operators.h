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
  int32_t block_shift;         // log2(block_size)
  uint32_t div_mul;            // row / (heads * parts) as a product: (row * div_mul >> 32) >> div_shift
  int32_t div_shift;           // -1: the divisor is 1
};
cudaError_t launch_paged_store(const PagedStoreParams& p, int row_type, int head_dim, int sms, cudaStream_t stream);

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
  int32_t bt_stride;
  int32_t num_blocks;
  // the cache's strides in units of `unit` bytes, the largest power of two
  // that divides them all: a token's offset is a 32-bit number of units
  uint32_t unit, block_units, head_units, tok_units;
  int32_t scale_off;                                        // bytes from a page to its scales
  int32_t heads, kv_heads, group;                           // group: query heads per key head
  int32_t next_n;                                           // prefill: 1
  int32_t k, max_blocks, block_size, block_shift, n_req;
  float scale_log2;                                         // softmax_scale * log2(e)
  int32_t head_chunks;          // chunks of attn_pad(group) heads that share a key head
  int32_t units;                // rows * kv_heads * head_chunks
  int32_t tiles;                // 128-entry tiles per row
};
// (tested ranges: the top-k's largest k, and the largest group in use; no
// buffer depends on either)
constexpr int kAttnMaxK = 2048;
constexpr int kAttnMaxGroup = 128;
constexpr int kAttnMaxCtas = 8;   // CTAs per unit (portable cluster size)
constexpr int kAttnTile = 128;    // selected tokens per MMA tile (MMA M of the scores, K of the outputs)
// Query heads of a unit, padded; a larger group is several units, each with
// its own copy of the tiles (64 heads' sums would not fit in the registers).
__host__ __device__ constexpr int attn_pad(int group) { return group <= 16 ? 16 : 32; }
// Roles: two epilogue warpgroups, each with four producer warps and a warp that
// issues its products; two query warps (register shares go by groups of four
// warps).
constexpr int kAttnGroups = 2;
constexpr int kAttnThreads = 32 * (4 * kAttnGroups + 4 * kAttnGroups + kAttnGroups + 2);
// Registers a thread after the launch's 96 have been dealt anew:
// 256 * 144 + 384 * 64 = 640 * 96.
constexpr int kAttnEpilogueRegs = 144, kAttnOtherRegs = 64;
// Probability buffers of a group: one is multiplied with the values while the
// next is written.
constexpr int kAttnProbBuffers = 2;
// Query buffers: the units in work and the next one (filled in the units'
// order, whichever pipeline they are for).
constexpr int kAttnQueryBuffers = kAttnGroups + 1;
// Tiles in flight, half of them a group's.  head_dim 128: a key
// half of a stage is free once its scores are computed, a value half only
// after the softmax and the output MMA, so they are rings of their own;
// head_dim 64 keeps both in one row of 128 bytes.  As many as fit next to
// the queries and probabilities.
constexpr uint32_t kAttnHalfBytes = kAttnTile * 128u;
__host__ __device__ constexpr int attn_k_stages(int head_dim) { return head_dim == 128 ? 4 : 0; }
__host__ __device__ constexpr int attn_v_stages(int head_dim) { return head_dim == 64 ? 8 : 6; }
struct AttnSmem {
  uint32_t k, v, q, p, scale, mask, flt, bars, misc, total;
};
// Floats of the softmax state of one CTA, GP heads (AttnState in sparse_attn.cu).
__host__ __device__ constexpr int attn_state_floats(int gp) { return 25 * gp + 40; }
__host__ __device__ constexpr AttnSmem attn_smem_layout(int head_dim, int gp) {
  AttnSmem L{};
  const uint32_t stages = static_cast<uint32_t>(attn_v_stages(head_dim));
  uint32_t off = 0;
  L.k = off;     off += attn_k_stages(head_dim) * kAttnHalfBytes;
  L.v = off;     off += stages * kAttnHalfBytes;
  L.q = off;     off += kAttnQueryBuffers * 2u * gp * 128u;  // 2*gp rows of 128 bytes
  L.p = off;     off += kAttnGroups * kAttnProbBuffers * kAttnTile * 2u * gp;  // tiles of probabilities
  L.scale = off; off += stages * kAttnTile * 8u;
  L.mask = off;  off += stages * 16u;
  L.flt = off;   off += 4u * attn_state_floats(gp);
  off = (off + 15u) & ~15u;
  L.bars = off;  off += 8u * 48u;
  L.misc = off;  off += 32u;
  L.total = off + 1024u;
  return L;
}
// ctas 0: persistent CTAs, a unit per epilogue group; 1 .. 8: a cluster of so
// many CTAs per unit, which share its tiles.
cudaError_t launch_sparse_attn(const SparseAttnParams& p, int head_dim, int grid, int ctas,
                               int smem_bytes, cudaStream_t stream);
cudaError_t read_attn_watchdog(unsigned int* value, bool clear);

}  // namespace fp8idx
