// Parameter blocks and launchers of the operators around the indexer: the
// step tables, the norms and rotations of the heads, the quantising paged
// stores, the sparse and the dense attention.
#pragma once

#include <cstdint>
#include <cuda.h>
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

// ------------------------------------------------- head norms and rotation
enum HeadNorm : int { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
constexpr int kNormRopeMaxDim = 256;
struct NormRopeParams {
  const void* x[2];            // queries, keys (or null)
  void* y[2];
  int64_t x_token[2], x_head[2], y_token[2], y_head[2];  // bytes
  const int32_t* positions;
  const float* inv_freq;
  const float* weight[2];      // or null
  const float* bias[2];        // or null
  int32_t tokens, dim, rot, rot_start, norm;
  int32_t heads[2];
  float eps, inv_dim, rope_scale;
  // set by the launcher: groups of heads side by side, how many of them a warp
  // walks, and warps per token
  int32_t groups[2], per, chunks;
};
cudaError_t launch_norm_rope(NormRopeParams& p, int row_type, bool pairs, int sms, cudaStream_t stream);

// ----------------------------------------------------- block-scaled store
struct BlockStoreParams {
  const void* x[2];            // keys, values
  int64_t token_stride[2];     // bytes
  int64_t head_stride[2];      // bytes
  const int32_t* slots;
  uint8_t* cache;
  int64_t block_stride;        // bytes between blocks
  int64_t cache_head_stride;   // bytes between heads
  int32_t num_slots, tokens, heads, block_shift;
  int32_t window;              // set by the launcher: rows of a CTA
};
cudaError_t launch_block_store(BlockStoreParams& p, int row_type, int head_dim, int sms, cudaStream_t stream);

// --------------------------------------------------------- dense attention
// A unit that several CTAs share, by the CTA that has its first piece.
struct BlockAttnMeta {
  int32_t row0, positions;     // first row; rows / heads per key head (0: no unit)
  int32_t head;                // key head
  int32_t last;                // CTA of the last piece
  int32_t shared;              // rows in two tiles of 128 lanes
  int32_t pad[3];
};
struct BlockAttnParams {
  const void* q;
  void* out;
  float* lse;                  // [rows][heads] or null
  const uint8_t* kv;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_new;       // [n_req + 1]
  float* partial;              // workspace: two pieces a CTA
  BlockAttnMeta* meta;         // workspace: one a CTA
  int64_t block_stride, head_stride;                                     // bytes
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;  // elements
  int64_t bt_stride;
  int32_t rows, heads, kv_heads, group;  // group: query heads per key head
  int32_t half_positions;      // positions of 128 lanes: 128 / group
  int32_t block_shift, max_blocks, num_blocks, n_req;
  int32_t window;              // positions a row sees, its own included (0: all)
  int32_t negative;            // the softmax scale's sign
  float scale_log2;            // |softmax_scale| * log2(e)
};
constexpr int kBlockAttnMaxGroup = 128;
// Partial results of rows whose positions several CTAs share: at most two
// pieces a CTA (one that began in an earlier CTA, one that ends in a later
// one), of 256 rows with D outputs, a reference, a sum and a scale each.
constexpr int kBlockAttnMaxCtas = 160, kBlockAttnLanes = 256;
__host__ __device__ constexpr int block_attn_piece_floats(int head_dim) { return kBlockAttnLanes * (head_dim + 4); }
constexpr size_t block_attn_workspace(int head_dim) {
  return static_cast<size_t>(kBlockAttnMaxCtas) * (2 * 4 * block_attn_piece_floats(head_dim) + sizeof(BlockAttnMeta));
}
// tm: the cache as [block][head][token][2 * head_dim bytes], boxes of a block's
// tokens by 128 bytes, 128-byte swizzle.
cudaError_t launch_block_attn(const CUtensorMap& tm, const BlockAttnParams& p, int head_dim, int grid, cudaStream_t stream);
int block_attn_smem(int head_dim);
cudaError_t read_block_attn_watchdog(unsigned int* value, bool clear);

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
