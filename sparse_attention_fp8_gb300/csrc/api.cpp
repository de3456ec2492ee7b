// C-ABI entry points of libfp8idx: argument validation, the host planner,
// TMA tensor-map encoding and kernel launch.  No allocation, no host
// synchronisation on the compute paths (both are graph-capturable).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "fp8idx.h"
#include "kernels.h"
#include "operators.h"

namespace {

using namespace fp8idx;

thread_local std::string g_last_error;

fp8idx_status fail(fp8idx_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

fp8idx_status ok() { return FP8IDX_OK; }

// ---------------------------------------------------------- device facts
struct DeviceInfo {
  int sms = 0;
  int smem_optin = 0;
  bool valid = false;
};
constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

fp8idx_status device_info(DeviceInfo* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "cudaGetDevice failed");
  if (dev < 0 || dev >= kMaxDevices) return fail(FP8IDX_ERR_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.valid) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return fail(FP8IDX_ERR_CUDA, "cudaDeviceGetAttribute failed");
    if (major != 10 || minor != 3)
      return fail(FP8IDX_ERR_UNSUPPORTED, "built for sm_103a; device is sm_%d%d", major, minor);
    d.valid = true;
  }
  *out = d;
  return FP8IDX_OK;
}

// ------------------------------------------ per-kernel shared-memory limit
struct SmemAttr {
  const void* kernel;
  int device;
  int bytes;
};
constexpr int kMaxSmemAttrs = 256;
SmemAttr g_smem_attr[kMaxSmemAttrs];
int g_smem_attr_n = 0;
std::mutex g_smem_attr_mu;

}  // namespace

namespace fp8idx {

// Sets the message fp8idx_last_error() returns on this thread (for entry
// points defined in other translation units).
void set_last_error_message(const char* msg) { g_last_error = msg; }

cudaError_t ensure_dynamic_smem(const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_smem_attr_mu);
  SmemAttr* hit = nullptr;
  for (int i = 0; i < g_smem_attr_n; ++i)
    if (g_smem_attr[i].kernel == kernel && g_smem_attr[i].device == dev) hit = &g_smem_attr[i];
  if (hit != nullptr && hit->bytes >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if (hit != nullptr) {
    hit->bytes = bytes;
  } else if (g_smem_attr_n < kMaxSmemAttrs) {
    g_smem_attr[g_smem_attr_n++] = SmemAttr{kernel, dev, bytes};
  }
  return cudaSuccess;
}

}  // namespace fp8idx

namespace {

using namespace fp8idx;

// ---------------------------------------------------- tensor-map encoding
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

fp8idx_status encode(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides_bytes, const uint32_t* box, CUtensorMapSwizzle swz, const char* what) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8IDX_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t gd[5], gs[5];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) {
    gd[i] = dims[i];
    bx[i] = box[i];
    es[i] = 1;
    if (i < rank - 1) gs[i] = strides_bytes[i];
  }
  CUresult r = fn(m, dt, static_cast<cuuint32_t>(rank), const_cast<void*>(base), gd, gs, bx, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FP8IDX_ERR_CUDA, "tensor map for %s: cuTensorMapEncodeTiled error %d", what, (int)r);
  return FP8IDX_OK;
}

// ------------------------------------------------------------ validation
int element_bytes(int dtype) { return dtype == FP8IDX_U8 ? 1 : (dtype == FP8IDX_BF16 || dtype == FP8IDX_F16) ? 2 : 4; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fp8idx_status check_tensor(const fp8idx_tensor* t, const char* name, int dtype, int ndim) {
  if (!t) return fail(FP8IDX_ERR_INVALID, "%s: null descriptor", name);
  if (t->ndim != ndim) return fail(FP8IDX_ERR_INVALID, "%s: ndim %d, expected %d", name, t->ndim, ndim);
  if (t->dtype != dtype) return fail(FP8IDX_ERR_INVALID, "%s: wrong dtype %d", name, t->dtype);
  int64_t numel = 1;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return fail(FP8IDX_ERR_INVALID, "%s: negative extent", name);
    numel *= t->shape[i];
  }
  if (numel > 0 && !t->data) return fail(FP8IDX_ERR_INVALID, "%s: null data pointer", name);
  if (numel > 0 && reinterpret_cast<uintptr_t>(t->data) % element_bytes(dtype) != 0)
    return fail(FP8IDX_ERR_INVALID, "%s: data is not aligned to its elements", name);
  return FP8IDX_OK;
}

bool contiguous(const fp8idx_tensor* t) {
  int64_t expect = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] != 1 && t->stride[i] != expect) return false;
    expect *= t->shape[i];
  }
  return true;
}

#define TRY(expr)                          \
  do {                                     \
    fp8idx_status _st = (expr);            \
    if (_st != FP8IDX_OK) return _st;      \
  } while (0)

// ---------------------------------------------------------------- planner

bool paged_supported(int heads, int head_dim, int block_size, int next_n) {
  if (head_dim != kHeadDim) return false;
  if (heads != 32 && heads != 64) return false;
  if (next_n < 1 || next_n * heads > 256) return false;
  return block_size == 1 || block_size == 16 || block_size == 32 || block_size == 64 || block_size == 128;
}

bool prefill_supported(int heads, int head_dim) {
  return (head_dim == kHeadDim || head_dim == 64) && (heads == 32 || heads == 64 || heads == 128);
}

fp8idx_status plan_paged(int32_t batch, int32_t next_n, int32_t heads, int32_t head_dim, int32_t block_size,
                         int32_t max_model_len, int32_t num_sms, int32_t smem_limit, const fp8idx_options* o,
                         fp8idx_plan* plan) {
  if (!paged_supported(heads, head_dim, block_size, next_n))
    return fail(FP8IDX_ERR_UNSUPPORTED, "decode: heads=%d head_dim=%d block_size=%d next_n=%d not supported", heads,
                head_dim, block_size, next_n);
  if (batch < 0 || batch > kMaxBatch) return fail(FP8IDX_ERR_UNSUPPORTED, "decode: batch %d > %d", batch, kMaxBatch);
  if (num_sms <= 0) return fail(FP8IDX_ERR_INVALID, "num_sms must be positive");
  const bool gather = block_size == 1;
  const int n_cols = next_n * heads;
  const int sub = paged_sub_tiles(n_cols, gather);
  int stages = (o && o->stages > 0) ? o->stages : 12 / sub;  // stages hold `sub` 128-token tiles each
  const int min_stages = gather ? 6 : 2;
  while (stages > min_stages && (int)paged_smem_layout(n_cols, stages, batch, sub).total > smem_limit) --stages;
  if (stages < min_stages || (int)paged_smem_layout(n_cols, stages, batch, sub).total > smem_limit)
    return fail(FP8IDX_ERR_UNSUPPORTED, "decode: shared memory too small for %d stages", stages);
  // Upper bound on work items without reading context_lens: every request
  // full to max_model_len.  The persistent grid never exceeds the SM count.
  const int64_t item_tokens = static_cast<int64_t>(kTileTokens) * sub;
  const int64_t tiles_per_req = (static_cast<int64_t>(std::max(max_model_len, 0)) + item_tokens - 1) / item_tokens;
  const int64_t items_ub = static_cast<int64_t>(batch) * tiles_per_req;
  int grid = static_cast<int>(std::min<int64_t>(num_sms, std::max<int64_t>(items_ub, 1)));
  if (o && o->num_ctas > 0) grid = std::min(o->num_ctas, num_sms);
  std::memset(plan, 0, sizeof(*plan));
  plan->grid = grid;
  plan->threads = paged_threads(gather);
  plan->smem_bytes = (int)paged_smem_layout(n_cols, stages, batch, sub).total;
  plan->stages = stages;
  plan->tile_n = n_cols;
  plan->block_m = next_n;
  plan->split_n = 1;
  plan->reverse_rows = 0;
  plan->tmem_cols = 512;
  plan->gather = gather ? 1 : 0;
  return FP8IDX_OK;
}

fp8idx_status plan_prefill(int64_t rows, int64_t cols, int32_t heads, int32_t head_dim, int32_t num_sms,
                           int32_t smem_limit, const fp8idx_options* o, fp8idx_plan* plan, int cu_entries = 0,
                           int min_stages = 2) {
  if (!prefill_supported(heads, head_dim))
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: heads=%d head_dim=%d not supported", heads, head_dim);
  if (rows < 0 || cols < 0 || rows * heads >= (1ll << 31) || cols >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: M=%lld N=%lld out of range", (long long)rows, (long long)cols);
  if (num_sms <= 0) return fail(FP8IDX_ERR_INVALID, "num_sms must be positive");
  int block_m = (o && o->block_m > 0) ? o->block_m : 256 / heads;
  if (block_m * heads > 256 || block_m > 32)
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: block_m %d too large for %d heads", block_m, heads);
  const int n_cols = block_m * heads;
  int stages = (o && o->stages > 0) ? o->stages : 12;
  while (stages > min_stages && (int)prefill_smem_layout(n_cols, stages, cu_entries, head_dim).total > smem_limit)
    --stages;
  if (stages < min_stages)
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: %d stages (this K source needs at least %d)", stages, min_stages);
  if ((int)prefill_smem_layout(n_cols, stages, cu_entries, head_dim).total > smem_limit)
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: shared memory too small");
  const int64_t num_rb = (rows + block_m - 1) / block_m;
  const int64_t n_tiles = (cols + kTileTokens - 1) / kTileTokens;
  int64_t split = 1;
  if (o && o->split_n > 0) {
    split = o->split_n;
  } else if (num_rb > 0) {
    // about 16 work units per persistent CTA keeps the round-robin deal
    // within a few percent of even
    split = (16ll * num_sms + num_rb - 1) / num_rb;
  }
  split = std::max<int64_t>(1, std::min<int64_t>(split, std::max<int64_t>(n_tiles, 1)));
  int reverse = (cols > 2048) ? 1 : 0;  // longest-first pays off only for long rows
  if (o && o->reverse_rows >= 0 && o->reverse_rows <= 1) reverse = o->reverse_rows;
  const int64_t units = num_rb * split;
  if (units > 0x7fffffffll) return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: too many work units");
  int grid = (int)std::min<int64_t>(num_sms, std::max<int64_t>(units, 1));
  if (o && o->num_ctas > 0) grid = std::min(o->num_ctas, num_sms);
  std::memset(plan, 0, sizeof(*plan));
  plan->grid = grid;
  plan->threads = prefill_threads();
  plan->smem_bytes = (int)prefill_smem_layout(n_cols, stages, cu_entries, head_dim).total;
  plan->stages = stages;
  plan->tile_n = n_cols;
  plan->block_m = block_m;
  plan->split_n = static_cast<int32_t>(split);
  plan->reverse_rows = reverse;
  plan->tmem_cols = 512;
  plan->gather = 0;
  return FP8IDX_OK;
}

// ----------------------------------------------------------------- decode
// Everything a decode launch needs except its output: the inputs checked,
// the plan, the tensor maps and the parameter block.
struct PagedSetup {
  CUtensorMap tm_q, tm_kv, tm_sc;
  PagedParams p;
  fp8idx_plan plan;
  int heads = 0;
  bool empty = false;  // nothing to compute (no requests or max_model_len 0)
};

fp8idx_status paged_setup(const fp8idx_tensor* q, const fp8idx_tensor* kv, const fp8idx_tensor* w,
                          const fp8idx_tensor* cl, const fp8idx_tensor* bt, int32_t max_model_len,
                          const fp8idx_options* opts, PagedSetup* S) {
  TRY(check_tensor(q, "q_fp8", FP8IDX_U8, 4));
  TRY(check_tensor(kv, "kv_cache", FP8IDX_U8, 2));
  TRY(check_tensor(w, "weights", FP8IDX_F32, 2));
  TRY(check_tensor(cl, "context_lens", FP8IDX_I32, 1));
  TRY(check_tensor(bt, "block_tables", FP8IDX_I32, 2));
  const int64_t B = q->shape[0], next_n = q->shape[1], H = q->shape[2], D = q->shape[3];
  if (max_model_len < 0) return fail(FP8IDX_ERR_INVALID, "max_model_len < 0");
  if (max_model_len > kMaxModelLen)
    return fail(FP8IDX_ERR_UNSUPPORTED, "max_model_len %d > %d (positions are kept in 32 bits)", max_model_len,
                kMaxModelLen);
  if (!contiguous(q)) return fail(FP8IDX_ERR_INVALID, "q_fp8 must be contiguous");
  if (!contiguous(kv)) return fail(FP8IDX_ERR_INVALID, "kv_cache must be contiguous");
  if (!contiguous(w)) return fail(FP8IDX_ERR_INVALID, "weights must be contiguous");
  if (cl->shape[0] != B || (B > 1 && cl->stride[0] != 1)) return fail(FP8IDX_ERR_INVALID, "context_lens must be [batch] contiguous");
  if (w->shape[0] != B * next_n || w->shape[1] != H) return fail(FP8IDX_ERR_INVALID, "weights must be [batch*next_n, heads]");
  if (bt->shape[0] != B || (bt->shape[1] > 1 && bt->stride[1] != 1) || (B > 1 && bt->stride[0] < bt->shape[1]))
    return fail(FP8IDX_ERR_INVALID, "block_tables must be [batch, max_blocks] with unit inner stride");
  if (D <= 0 || kv->shape[1] % (D + 4) != 0) return fail(FP8IDX_ERR_INVALID, "kv_cache row is not block_size*(head_dim+4) bytes");
  const int64_t blk = kv->shape[1] / (D + 4);
  if (next_n <= 0 || H <= 0 || blk <= 0) return fail(FP8IDX_ERR_INVALID, "empty next_n/heads/block_size");
  if (!paged_supported((int)H, (int)D, (int)blk, (int)next_n))
    return fail(FP8IDX_ERR_UNSUPPORTED, "decode: heads=%lld head_dim=%lld block_size=%lld next_n=%lld not supported",
                (long long)H, (long long)D, (long long)blk, (long long)next_n);
  S->empty = B == 0 || max_model_len == 0;
  if (S->empty) return ok();
  if (kv->shape[0] < 1) return fail(FP8IDX_ERR_INVALID, "kv_cache has no blocks");
  if (bt->shape[1] < 1) return fail(FP8IDX_ERR_INVALID, "block_tables has no columns");
  if (!aligned16(q->data) || !aligned16(kv->data) || !aligned16(w->data))
    return fail(FP8IDX_ERR_INVALID, "q_fp8, kv_cache and weights must be 16-byte aligned");
  if (B * next_n * H >= (1ll << 31) || kv->shape[0] >= (1ll << 31) || bt->shape[1] >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "decode: extents too large");

  DeviceInfo dev;
  TRY(device_info(&dev));
  fp8idx_plan& plan = S->plan;
  TRY(plan_paged((int)B, (int)next_n, (int)H, (int)D, (int)blk, max_model_len, dev.sms, dev.smem_optin, opts, &plan));

  const int n_cols = (int)(next_n * H);
  {
    const uint64_t dims[2] = {(uint64_t)D, (uint64_t)(B * n_cols)};
    const uint64_t strides[1] = {(uint64_t)D};
    const uint32_t box[2] = {(uint32_t)D, (uint32_t)n_cols};
    TRY(encode(&S->tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q->data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
               "q"));
  }
  if (!plan.gather) {
    // K rows: [block][row][128 B]; scales: [block][blk f32], starting after the block's K rows
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)blk, (uint64_t)kv->shape[0]};
    const uint64_t strides[2] = {(uint64_t)D, (uint64_t)kv->shape[1]};
    const uint32_t box[3] = {(uint32_t)D, (uint32_t)blk, 1u};
    TRY(encode(&S->tm_kv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, kv->data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
               "kv_cache"));
    const uint64_t sdims[2] = {(uint64_t)blk, (uint64_t)kv->shape[0]};
    const uint64_t sstrides[1] = {(uint64_t)kv->shape[1]};
    const uint32_t sbox[2] = {(uint32_t)blk, 1u};
    TRY(encode(&S->tm_sc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, static_cast<const uint8_t*>(kv->data) + blk * D, sdims,
               sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE, "kv_cache scales"));
  } else {
    S->tm_kv = S->tm_q;  // unused by the gather kernel
    S->tm_sc = S->tm_q;
  }
  PagedParams& p = S->p;
  std::memset(&p, 0, sizeof(p));
  p.kv_cache = static_cast<const uint8_t*>(kv->data);
  p.weights = static_cast<const float*>(w->data);
  p.context_lens = static_cast<const int32_t*>(cl->data);
  p.block_tables = static_cast<const int32_t*>(bt->data);
  p.bt_stride = B > 1 ? bt->stride[0] : bt->shape[1];
  p.num_blocks = kv->shape[0];
  p.batch = (int32_t)B;
  p.next_n = (int32_t)next_n;
  p.max_blocks = (int32_t)bt->shape[1];
  p.max_model_len = max_model_len;
  p.block_size = (int32_t)blk;
  p.n_cols = n_cols;
  p.stages = plan.stages;
  p.sub_tiles = paged_sub_tiles(n_cols, plan.gather != 0);
  p.acc_bufs = paged_acc_buffers(n_cols, p.sub_tiles);
  S->heads = (int)H;
  return ok();
}

// mode: 0 the logits, 1 the fused top-k's filter pass, 2 its sample pass
fp8idx_status paged_launch(const PagedSetup& S, const PagedParams& p, int mode, void* stream) {
  cudaError_t e = launch_paged(S.tm_q, S.tm_kv, S.tm_sc, p, S.heads, S.plan.gather != 0, S.plan.grid,
                               S.plan.smem_bytes, static_cast<cudaStream_t>(stream), mode);
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
  return ok();
}

fp8idx_status paged_impl(const fp8idx_tensor* q, const fp8idx_tensor* kv, const fp8idx_tensor* w,
                         const fp8idx_tensor* cl, const fp8idx_tensor* bt, int32_t max_model_len,
                         const fp8idx_tensor* out, const fp8idx_options* opts, void* stream) {
  g_last_error.clear();
  TRY(check_tensor(q, "q_fp8", FP8IDX_U8, 4));
  TRY(check_tensor(kv, "kv_cache", FP8IDX_U8, 2));
  TRY(check_tensor(w, "weights", FP8IDX_F32, 2));
  TRY(check_tensor(cl, "context_lens", FP8IDX_I32, 1));
  TRY(check_tensor(bt, "block_tables", FP8IDX_I32, 2));
  TRY(check_tensor(out, "out", FP8IDX_F32, 2));
  const int64_t B = q->shape[0], next_n = q->shape[1];
  if (max_model_len < 0) return fail(FP8IDX_ERR_INVALID, "max_model_len < 0");
  if (out->shape[0] != B * next_n || out->shape[1] < max_model_len ||
      (out->shape[1] > 1 && out->stride[1] != 1) || (out->shape[0] > 1 && out->stride[0] < out->shape[1]))
    return fail(FP8IDX_ERR_INVALID, "out must be [batch*next_n, >=max_model_len] with unit inner stride");
  PagedSetup S;
  TRY(paged_setup(q, kv, w, cl, bt, max_model_len, opts, &S));
  if (S.empty) return ok();
  PagedParams p = S.p;
  p.out = static_cast<float*>(out->data);
  p.out_stride = out->shape[0] > 1 ? out->stride[0] : out->shape[1];
  return paged_launch(S, p, 0, stream);
}

// ----------------------------------------------------- fused decode top-k
// fp8_paged_mqa_topk: six launches on the caller's stream, none of which
// writes the logits of every row:
//   1. the decode kernel on every 32nd item of each request, its logits into
//      the workspace (the threshold sample);
//   2. per row: reset of the row's state, the threshold;
//   3. the decode kernel in its filter form: per row only the logits at or
//      above the threshold, with a bitmap of their positions, instead of
//      every logit;
//   4. per row: the exact top-k from the candidates, or the row flagged;
//   5. the decode kernel over the flagged requests only, all their logits
//      into the workspace, and 6. the top-k kernel over the flagged rows --
//      both return at once when no row was flagged.
size_t paged_topk_workspace(int64_t batch, int64_t next_n, int64_t max_model_len, int32_t k) {
  return static_cast<size_t>(fused_topk_layout(batch, next_n, max_model_len, k).total);
}

fp8idx_status paged_topk_impl(const fp8idx_tensor* q, const fp8idx_tensor* kv, const fp8idx_tensor* w,
                              const fp8idx_tensor* cl, const fp8idx_tensor* bt, int32_t max_model_len, int32_t k,
                              const fp8idx_tensor* indices, void* workspace, size_t workspace_bytes,
                              const fp8idx_options* opts, void* stream) {
  g_last_error.clear();
  TRY(check_tensor(q, "q_fp8", FP8IDX_U8, 4));
  TRY(check_tensor(indices, "indices", FP8IDX_I32, 2));
  const int64_t B = q->shape[0], next_n = q->shape[1], R = B * next_n;
  if (k < 1 || k > kTopkMaxK) return fail(FP8IDX_ERR_UNSUPPORTED, "top-k: k=%d not in [1, %d]", k, kTopkMaxK);
  if (max_model_len < 0) return fail(FP8IDX_ERR_INVALID, "max_model_len < 0");
  if (indices->shape[0] != R || indices->shape[1] != k || (k > 1 && indices->stride[1] != 1) ||
      (R > 1 && indices->stride[0] < k))
    return fail(FP8IDX_ERR_INVALID, "indices must be [batch*next_n, k] with unit inner stride");
  PagedSetup S;
  TRY(paged_setup(q, kv, w, cl, bt, max_model_len, opts, &S));
  if (R == 0) return ok();
  const FusedTopkLayout L = fused_topk_layout(B, next_n, max_model_len, k);
  if (workspace == nullptr || workspace_bytes < L.total)
    return fail(FP8IDX_ERR_INVALID, "workspace of %zu bytes, %llu needed (fp8idx_paged_mqa_topk_workspace)",
                workspace_bytes, (unsigned long long)L.total);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(FP8IDX_ERR_INVALID, "workspace must be 256-byte aligned");
  if (R >= (1ll << 31) / kTopkMaxCluster) return fail(FP8IDX_ERR_UNSUPPORTED, "top-k: too many rows");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FusedTopkParams f;
  std::memset(&f, 0, sizeof(f));
  f.context_lens = static_cast<const int32_t*>(cl->data);
  f.rows = (int32_t)R;
  f.next_n = (int32_t)next_n;
  f.cols = max_model_len;
  f.k = k;
  f.logits = reinterpret_cast<float*>(ws + L.logits);
  f.ls = L.ls;
  f.tw = L.tw;
  f.thr = reinterpret_cast<float*>(ws + L.thr);
  f.cand = reinterpret_cast<uint32_t*>(ws + L.cand);
  f.req_flag = reinterpret_cast<uint32_t*>(ws + L.req_flag);
  f.row_flag = reinterpret_cast<uint32_t*>(ws + L.row_flag);
  f.any = reinterpret_cast<uint32_t*>(ws + L.any);
  f.out = static_cast<int32_t*>(indices->data);
  f.out_stride = R > 1 ? indices->stride[0] : k;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (S.empty) {  // max_model_len 0: every window is empty
    f.item_tokens = kTileTokens;
    cudaError_t e = launch_fused_threshold(f, fused_threshold_smem_bytes(), st);
    if (e == cudaSuccess) e = launch_fused_select(f, fused_select_smem_bytes(), st);
    if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "top-k launch: %s", cudaGetErrorString(e));
    return ok();
  }
  f.item_tokens = kTileTokens * S.p.sub_tiles;

  // 1. the sample
  PagedParams p = S.p;
  p.out = f.logits;
  p.out_stride = L.ls;
  TRY(paged_launch(S, p, 2, stream));
  // 2. thresholds
  cudaError_t e = launch_fused_threshold(f, fused_threshold_smem_bytes(), st);
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "top-k threshold launch: %s", cudaGetErrorString(e));
  // 3. the filter pass
  p = S.p;
  p.out = f.logits;
  p.out_stride = L.ls;
  p.thr = f.thr;
  p.cand_bits = f.cand;
  p.bits_stride = L.tw;
  TRY(paged_launch(S, p, 1, stream));
  // 4. the exact selection, or the row flagged
  e = launch_fused_select(f, fused_select_smem_bytes(), st);
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "top-k select launch: %s", cudaGetErrorString(e));
  // 5. and 6. the exact fallback for flagged rows
  p = S.p;
  p.out = f.logits;
  p.out_stride = L.ls;
  p.req_mask = f.req_flag;
  p.run_flag = f.any;
  TRY(paged_launch(S, p, 0, stream));
  TopkParams tp;
  std::memset(&tp, 0, sizeof(tp));
  tp.mode = 1;
  tp.k = k;
  tp.rows = (int32_t)R;
  tp.context_lens = f.context_lens;
  tp.cols = max_model_len;
  tp.next_n = (int32_t)next_n;
  tp.logits = f.logits;
  tp.stride = L.ls;
  tp.out = f.out;
  tp.out_stride = f.out_stride;
  tp.vec_ok = 1;  // workspace rows are 16-byte aligned
  tp.row_mask = f.row_flag;
  tp.run_flag = f.any;
  DeviceInfo dev;
  TRY(device_info(&dev));
  int cap = kTopkMaxCap;
  while (cap > 1024 && (int)topk_smem_layout(cap).total > dev.smem_optin) cap >>= 1;
  tp.cap = cap;
  e = launch_topk(tp, 1, (int)topk_smem_layout(cap).total, st);
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "top-k fallback launch: %s", cudaGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- prefill
// The K source of a prefill call: contiguous (k, s) or paged (kv, bt, cu).
struct PrefillK {
  const fp8idx_tensor* k = nullptr;
  const fp8idx_tensor* s = nullptr;
  const fp8idx_tensor* kv = nullptr;
  const fp8idx_tensor* bt = nullptr;
  const fp8idx_tensor* cu = nullptr;
};

fp8idx_status prefill_impl(const fp8idx_tensor* q, const PrefillK& src, const fp8idx_tensor* w,
                           const fp8idx_tensor* ks, const fp8idx_tensor* ke, const fp8idx_tensor* out,
                           const fp8idx_options* opts, void* stream) {
  g_last_error.clear();
  const bool paged = src.kv != nullptr;
  TRY(check_tensor(q, "q_fp8", FP8IDX_U8, 3));
  TRY(check_tensor(w, "weights", FP8IDX_F32, 2));
  TRY(check_tensor(ks, "cu_seqlen_ks", FP8IDX_I32, 1));
  TRY(check_tensor(ke, "cu_seqlen_ke", FP8IDX_I32, 1));
  TRY(check_tensor(out, "out", FP8IDX_F32, 2));
  const int64_t M = q->shape[0], H = q->shape[1], D = q->shape[2];
  int64_t N = 0, blk = 0, R = 0;
  if (!paged) {
    TRY(check_tensor(src.k, "k_fp8", FP8IDX_U8, 2));
    TRY(check_tensor(src.s, "kv_scale", FP8IDX_F32, 1));
    N = src.k->shape[0];
    if (!contiguous(src.k) || !contiguous(src.s)) return fail(FP8IDX_ERR_INVALID, "prefill inputs must be contiguous");
    if (src.k->shape[1] != D || src.s->shape[0] != N)
      return fail(FP8IDX_ERR_INVALID, "k_fp8 must be [N, head_dim], kv_scale [N]");
  } else {
    TRY(check_tensor(src.kv, "kv_cache", FP8IDX_U8, 2));
    TRY(check_tensor(src.bt, "block_tables", FP8IDX_I32, 2));
    TRY(check_tensor(src.cu, "cu_seq_lens", FP8IDX_I32, 1));
    N = out->shape[1];
    R = src.bt->shape[0];
    if (!contiguous(src.kv) || !contiguous(src.cu)) return fail(FP8IDX_ERR_INVALID, "kv_cache and cu_seq_lens must be contiguous");
    if (src.bt->shape[1] > 1 && src.bt->stride[1] != 1) return fail(FP8IDX_ERR_INVALID, "block_tables rows must be contiguous");
    if (src.cu->shape[0] != R + 1) return fail(FP8IDX_ERR_INVALID, "cu_seq_lens must be [requests + 1]");
    if (D != kHeadDim && D != 64)
      return fail(FP8IDX_ERR_UNSUPPORTED, "paged prefill: head_dim %lld (128 or 64)", (long long)D);
    if (src.kv->shape[1] % (D + 4) != 0) return fail(FP8IDX_ERR_INVALID, "kv_cache rows must be block_size*(head_dim+4) bytes");
    blk = src.kv->shape[1] / (D + 4);
    if (blk != 1 && blk != 16 && blk != 32 && blk != 64 && blk != 128)
      return fail(FP8IDX_ERR_UNSUPPORTED, "paged prefill: block_size %lld not in {1, 16, 32, 64, 128}", (long long)blk);
    if (R < 1 || R > kMaxBatch) return fail(FP8IDX_ERR_UNSUPPORTED, "paged prefill: %lld requests (1..%d)", (long long)R, kMaxBatch);
    if (src.bt->shape[1] < 1 || src.kv->shape[0] < 1) return fail(FP8IDX_ERR_INVALID, "empty block table or cache");
    if (!aligned16(src.kv->data)) return fail(FP8IDX_ERR_INVALID, "kv_cache must be 16-byte aligned");
  }
  if (!contiguous(q) || !contiguous(w) || !contiguous(ks) || !contiguous(ke))
    return fail(FP8IDX_ERR_INVALID, "prefill inputs must be contiguous");
  if (w->shape[0] != M || w->shape[1] != H) return fail(FP8IDX_ERR_INVALID, "weights must be [M, heads]");
  if (ks->shape[0] != M || ke->shape[0] != M) return fail(FP8IDX_ERR_INVALID, "cu_seqlen_ks/ke must be [M]");
  if (out->shape[0] != M || out->shape[1] != N || (N > 1 && out->stride[1] != 1) || (M > 1 && out->stride[0] < N))
    return fail(FP8IDX_ERR_INVALID, "out must be [M, N] with unit inner stride");
  if (!prefill_supported((int)H, (int)D))
    return fail(FP8IDX_ERR_UNSUPPORTED, "prefill: heads=%lld head_dim=%lld not supported", (long long)H, (long long)D);
  if (M == 0 || N == 0) return ok();
  if (!aligned16(q->data) || !aligned16(w->data) || (!paged && (!aligned16(src.k->data) || !aligned16(src.s->data))))
    return fail(FP8IDX_ERR_INVALID, "q_fp8, k_fp8, kv_scale and weights must be 16-byte aligned");
  DeviceInfo dev;
  TRY(device_info(&dev));
  fp8idx_plan plan;
  // the block-size-1 token gather publishes tiles 4 behind: at least 6 stages
  TRY(plan_prefill(M, N, (int)H, (int)D, dev.sms, dev.smem_optin, opts, &plan, paged ? 2 * ((int)R + 1) : 0,
                   (paged && blk == 1) ? 6 : 2));
  CUtensorMap tm_q, tm_k, tm_s;
  {
    const uint64_t dims[2] = {(uint64_t)D, (uint64_t)(M * H)};
    const uint64_t strides[1] = {(uint64_t)D};
    const uint32_t box[2] = {(uint32_t)D, (uint32_t)plan.tile_n};
    TRY(encode(&tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q->data, dims, strides, box,
               D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, "q"));
  }
  std::memset(&tm_k, 0, sizeof(tm_k));
  std::memset(&tm_s, 0, sizeof(tm_s));
  if (paged && blk > 1) {  // (block size 1 is gathered per token with cp.async: no tensor maps)
    // K rows of the cache: [block][row][D bytes]; scales: [block][blk f32] after the block's K rows
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)blk, (uint64_t)src.kv->shape[0]};
    const uint64_t strides[2] = {(uint64_t)D, (uint64_t)src.kv->shape[1]};
    const uint32_t box[3] = {(uint32_t)D, (uint32_t)blk, 1u};
    TRY(encode(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, src.kv->data, dims, strides, box,
               D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, "kv_cache"));
    if (blk >= 32) {
      const uint64_t sdims[2] = {(uint64_t)blk, (uint64_t)src.kv->shape[0]};
      const uint64_t sstrides[1] = {(uint64_t)src.kv->shape[1]};
      const uint32_t sbox[2] = {(uint32_t)blk, 1u};
      TRY(encode(&tm_s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, static_cast<const uint8_t*>(src.kv->data) + blk * D,
                 sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE, "kv_cache scales"));
    }
  } else if (!paged) {
    {
      const uint64_t dims[2] = {(uint64_t)D, (uint64_t)N};
      const uint64_t strides[1] = {(uint64_t)D};
      const uint32_t box[2] = {(uint32_t)D, (uint32_t)kTileTokens};
      TRY(encode(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, src.k->data, dims, strides, box,
                 D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, "k"));
    }
    {
      const uint64_t dims[1] = {(uint64_t)N};
      const uint32_t box[1] = {(uint32_t)kTileTokens};
      TRY(encode(&tm_s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 1, src.s->data, dims, nullptr, box,
                 CU_TENSOR_MAP_SWIZZLE_NONE, "kv_scale"));
    }
  }
  CUtensorMap tm_w;
  {
    const uint64_t dims[1] = {(uint64_t)(M * H)};
    const uint32_t box[1] = {(uint32_t)plan.tile_n};
    TRY(encode(&tm_w, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 1, w->data, dims, nullptr, box, CU_TENSOR_MAP_SWIZZLE_NONE,
               "weights"));
  }
  PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  if (paged) {
    p.kv_cache = static_cast<const uint8_t*>(src.kv->data);
    p.block_tables = static_cast<const int32_t*>(src.bt->data);
    p.cu_seq_lens = static_cast<const int32_t*>(src.cu->data);
    p.bt_stride = R > 1 ? src.bt->stride[0] : src.bt->shape[1];
    p.num_blocks = src.kv->shape[0];
    p.max_blocks = (int32_t)src.bt->shape[1];
    p.block_size = (int32_t)blk;
    p.n_req = (int32_t)R;
  }
  p.ks = static_cast<const int32_t*>(ks->data);
  p.ke = static_cast<const int32_t*>(ke->data);
  p.out = static_cast<float*>(out->data);
  p.out_stride = M > 1 ? out->stride[0] : N;
  p.rows = (int32_t)M;
  p.cols = (int32_t)N;
  p.block_m = plan.block_m;
  p.n_cols = plan.tile_n;
  p.stages = plan.stages;
  p.split = plan.split_n;
  p.reverse = plan.reverse_rows;
  p.vec_ok = (aligned16(out->data) && (p.out_stride % 4) == 0) ? 1 : 0;
  p.clean = (opts && opts->clean_logits < 0) ? 0 : 1;
  p.acc_bufs = paged_acc_buffers(plan.tile_n);
  // -inf tiles as TMA stores need 16-byte aligned rows (the tensor map's
  // stride rule); otherwise the epilogue warps write them.  A TMA store
  // writes whole 16-byte units, so the map is N rounded down to a multiple
  // of 4 columns wide and the kernel writes the rest of the row directly.
  CUtensorMap tm_out;
  std::memset(&tm_out, 0, sizeof(tm_out));
  p.tma_fill = 0;
  p.fill_cols = (int32_t)(N & ~3ll);
  if (p.clean && p.vec_ok && p.fill_cols > 0) {
    const uint64_t dims[2] = {(uint64_t)p.fill_cols, (uint64_t)M};
    const uint64_t strides[1] = {(uint64_t)p.out_stride * 4u};
    const uint32_t box[2] = {(uint32_t)kTileTokens, (uint32_t)plan.block_m};
    TRY(encode(&tm_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, out->data, dims, strides, box,
               CU_TENSOR_MAP_SWIZZLE_NONE, "out"));
    p.tma_fill = 1;
  }
  cudaError_t e = launch_prefill(tm_q, tm_k, tm_s, tm_w, tm_out, p, (int)H, (int)D, paged, plan.grid, plan.smem_bytes,
                                 static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
  return ok();
}

// ------------------------------------------------------------------ top-k
// mode 0: prefill windows from ks/ke over the row width; mode 1: decode
// windows from context_lens/next_n within max_model_len columns.
fp8idx_status topk_impl(int mode, const fp8idx_tensor* logits, const fp8idx_tensor* ks, const fp8idx_tensor* ke,
                        const fp8idx_tensor* cl, int32_t next_n, int32_t max_model_len, int32_t k,
                        const fp8idx_tensor* indices, const fp8idx_options* opts, void* stream) {
  g_last_error.clear();
  TRY(check_tensor(logits, "logits", FP8IDX_F32, 2));
  TRY(check_tensor(indices, "indices", FP8IDX_I32, 2));
  const int64_t R = logits->shape[0], W = logits->shape[1];
  if (k < 1 || k > kTopkMaxK) return fail(FP8IDX_ERR_UNSUPPORTED, "top-k: k=%d not in [1, %d]", k, kTopkMaxK);
  if (W > 1 && logits->stride[1] != 1) return fail(FP8IDX_ERR_INVALID, "logits must have unit inner stride");
  if (R > 1 && logits->stride[0] < W) return fail(FP8IDX_ERR_INVALID, "logits rows overlap");
  if (indices->shape[0] != R || indices->shape[1] != k || (k > 1 && indices->stride[1] != 1) ||
      (R > 1 && indices->stride[0] < k))
    return fail(FP8IDX_ERR_INVALID, "indices must be [rows, k] with unit inner stride");
  if (W >= (1ll << 31) || R * kTopkMaxCluster >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "top-k: logits too large");
  const int32_t ctas_req = opts ? opts->num_ctas : 0;
  if (ctas_req < 0 || ctas_req > kTopkMaxCluster)
    return fail(FP8IDX_ERR_UNSUPPORTED, "top-k: num_ctas=%d not in [0, %d]", ctas_req, kTopkMaxCluster);
  TopkParams p;
  std::memset(&p, 0, sizeof(p));
  p.mode = mode;
  p.k = k;
  p.rows = (int32_t)R;
  if (mode == 0) {
    TRY(check_tensor(ks, "cu_seqlen_ks", FP8IDX_I32, 1));
    TRY(check_tensor(ke, "cu_seqlen_ke", FP8IDX_I32, 1));
    if (ks->shape[0] != R || ke->shape[0] != R || !contiguous(ks) || !contiguous(ke))
      return fail(FP8IDX_ERR_INVALID, "cu_seqlen_ks/ke must be contiguous [rows]");
    p.ks = static_cast<const int32_t*>(ks->data);
    p.ke = static_cast<const int32_t*>(ke->data);
    p.cols = (int32_t)W;
    p.next_n = 1;
  } else {
    TRY(check_tensor(cl, "context_lens", FP8IDX_I32, 1));
    if (next_n < 1) return fail(FP8IDX_ERR_INVALID, "next_n must be positive");
    if (!contiguous(cl) || cl->shape[0] * next_n != R)
      return fail(FP8IDX_ERR_INVALID, "context_lens must be contiguous [rows / next_n]");
    if (max_model_len < 0 || max_model_len > W)
      return fail(FP8IDX_ERR_INVALID, "max_model_len must be in [0, logits width]");
    p.context_lens = static_cast<const int32_t*>(cl->data);
    p.cols = max_model_len;
    p.next_n = next_n;
  }
  if (R == 0) return ok();
  p.logits = static_cast<const float*>(logits->data);
  p.stride = R > 1 ? logits->stride[0] : W;
  p.out = static_cast<int32_t*>(indices->data);
  p.out_stride = R > 1 ? indices->stride[0] : k;
  p.vec_ok = (aligned16(logits->data) && (p.stride % 4) == 0) ? 1 : 0;
  DeviceInfo dev;
  TRY(device_info(&dev));
  // CTAs per row: a cluster per row only when the rows leave most SMs idle
  // (at most a quarter of the SM count) and the longest possible window
  // gives each CTA at least kTopkMinSlice values; with more rows the
  // cluster's barriers cost more than the extra SMs return (measured).
  int ctas = 1;
  if (p.cols >= 2 * kTopkMinSlice && 4 * R <= dev.sms) {
    const int64_t by_rows = dev.sms / R, by_len = p.cols / kTopkMinSlice;
    ctas = (int)std::min<int64_t>(kTopkMaxCluster, std::min(by_rows, by_len));
    if (ctas < 2) ctas = 1;
  }
  if (ctas_req > 0) ctas = ctas_req;
  int cap = kTopkMaxCap;
  while (cap > 1024 && (int)topk_smem_layout(cap).total > dev.smem_optin) cap >>= 1;
  p.cap = cap;
  cudaError_t e = launch_topk(p, ctas, (int)topk_smem_layout(cap).total, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "top-k launch: %s", cudaGetErrorString(e));
  return ok();
}

// ------------------------------------------- the operators around the indexer
bool block_size_ok(int64_t bs) { return bs == 1 || bs == 16 || bs == 32 || bs == 64 || bs == 128; }
bool row_dim_ok(int64_t d) { return d == 64 || d == 128; }
int64_t kv_page_bytes(int64_t bs, int64_t d) { return (bs * (2 * d + 8) + 15) / 16 * 16; }
int64_t kv_block_page_bytes(int64_t bs, int64_t d) { return bs * 2 * d + 16; }

fp8idx_status check_vector(const fp8idx_tensor* t, const char* name, int64_t n) {
  TRY(check_tensor(t, name, FP8IDX_I32, 1));
  if (t->shape[0] != n || (n > 1 && t->stride[0] != 1))
    return fail(FP8IDX_ERR_INVALID, "%s: expected contiguous [%lld]", name, (long long)n);
  return FP8IDX_OK;
}

// The bytes of a tensor with non-negative strides: runs of `run` bytes, spaced
// by the strides of the dimensions that are not part of a run (largest first;
// a stride of 0 repeats the same bytes).
struct Extent {
  uintptr_t at = 0;
  int64_t run = 0, size = 0;  // bytes of a run (0: empty), from the first byte to the last
  int dims = 0;
  int64_t count[4], stride[4];

  explicit Extent(const fp8idx_tensor* t) {
    at = reinterpret_cast<uintptr_t>(t->data);
    const int64_t item = element_bytes(t->dtype);
    run = item;
    for (int i = t->ndim - 1; i >= 0; --i) {
      if (t->shape[i] == 0) {
        run = size = 0;
        return;
      }
      if (t->shape[i] == 1 || t->stride[i] == 0) continue;
      const int64_t step = t->stride[i] * item;
      if (dims == 0 && step == run) {
        run *= t->shape[i];
        continue;
      }
      int j = dims++;
      for (; j > 0 && stride[j - 1] < step; --j) stride[j] = stride[j - 1], count[j] = count[j - 1];
      stride[j] = step;
      count[j] = t->shape[i];
    }
    size = run;
    for (int i = 0; i < dims; ++i) size += (count[i] - 1) * stride[i];
  }
  // One step of the outermost dimension, moved by `by` bytes.
  Extent inner(int64_t by) const {
    Extent e = *this;
    e.at += static_cast<uintptr_t>(by);
    e.size -= (count[0] - 1) * stride[0];
    --e.dims;
    for (int i = 0; i < e.dims; ++i) e.count[i] = count[i + 1], e.stride[i] = stride[i + 1];
    return e;
  }
  // Whether two elements share bytes.  (Exact for views of a tensor, whose
  // dimensions lie within one another.)
  bool overlaps_itself() const {
    int64_t within = run;
    for (int i = dims - 1; i >= 0; --i) {
      if (stride[i] < within) return true;
      within += (count[i] - 1) * stride[i];
    }
    return false;
  }
};

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }

// Whether two tensors share bytes.  Slices of one tensor that lie between one
// another do not.  Both are taken apart step by step, at most `budget` steps,
// after which they count as overlapping.
bool share_bytes(const Extent& a, const Extent& b, int* budget) {
  if (a.run == 0 || b.run == 0 || a.at >= b.at + static_cast<uintptr_t>(b.size) ||
      b.at >= a.at + static_cast<uintptr_t>(a.size))
    return false;
  if (a.dims == 0 && b.dims == 0) return true;
  if (a.dims == 0 || (b.dims > 0 && b.stride[0] > a.stride[0])) return share_bytes(b, a, budget);
  // the steps k of a's outermost dimension (with equal strides: the difference
  // of both's steps) that come near b
  const bool both = b.dims > 0 && b.stride[0] == a.stride[0];
  const Extent x = a.inner(0), y = both ? b.inner(0) : b;
  const int64_t s = a.stride[0], d = static_cast<int64_t>(y.at - x.at);
  const int64_t lo = std::max(floor_div(d - x.size, s) + 1, both ? 1 - b.count[0] : int64_t{0});
  const int64_t hi = std::min(floor_div(d + y.size - 1, s), a.count[0] - 1);
  for (int64_t k = lo; k <= hi; ++k)
    if (--*budget < 0 || share_bytes(a.inner(k * s), y, budget)) return true;
  return false;
}
bool tensors_overlap(const fp8idx_tensor* a, const fp8idx_tensor* b) {
  int budget = 1024;
  return share_bytes(Extent(a), Extent(b), &budget);
}

fp8idx_status step_tables_impl(const fp8idx_tensor* old_lens, const fp8idx_tensor* new_lens,
                               const fp8idx_tensor* free_blocks, const fp8idx_tensor* free_count, int32_t block_size,
                               const fp8idx_tensor* bt, const fp8idx_tensor* ctx, const fp8idx_tensor* cu_new,
                               const fp8idx_tensor* slots, const fp8idx_tensor* counts, const fp8idx_tensor* cu_seq,
                               const fp8idx_tensor* ks, const fp8idx_tensor* ke, void* stream) {
  g_last_error.clear();
  TRY(check_tensor(old_lens, "old_lens", FP8IDX_I32, 1));
  const int64_t B = old_lens->shape[0];
  TRY(check_vector(old_lens, "old_lens", B));
  TRY(check_vector(new_lens, "new_lens", B));
  TRY(check_tensor(free_blocks, "free_blocks", FP8IDX_I32, 1));
  TRY(check_vector(free_blocks, "free_blocks", free_blocks->shape[0]));
  TRY(check_vector(free_count, "free_count", 1));
  TRY(check_tensor(bt, "block_tables", FP8IDX_I32, 2));
  if (bt->shape[0] != B || (B > 0 && bt->shape[1] > 1 && bt->stride[1] != 1) ||
      (B > 1 && bt->stride[0] < bt->shape[1]))
    return fail(FP8IDX_ERR_INVALID, "block_tables must be [batch, max_blocks] with contiguous rows");
  TRY(check_vector(ctx, "context_lens", B));
  TRY(check_vector(cu_new, "cu_new_lens", B + 1));
  TRY(check_tensor(slots, "slot_mapping", FP8IDX_I32, 1));
  const int64_t T = slots->shape[0];
  TRY(check_vector(slots, "slot_mapping", T));
  TRY(check_vector(counts, "counts", 4));
  if (cu_seq) TRY(check_vector(cu_seq, "cu_seq_lens", B + 1));
  if (ks) TRY(check_vector(ks, "cu_seqlen_ks", T));
  if (ke) TRY(check_vector(ke, "cu_seqlen_ke", T));
  if (!block_size_ok(block_size))
    return fail(FP8IDX_ERR_UNSUPPORTED, "step tables: block_size %d not in {1, 16, 32, 64, 128}", block_size);
  if (B > kMaxBatch) return fail(FP8IDX_ERR_UNSUPPORTED, "step tables: batch %lld > %d", (long long)B, kMaxBatch);
  if (bt->shape[1] * block_size >= (1ll << 31) || T >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "step tables: positions and rows must stay below 2^31");
  const fp8idx_tensor* ins[] = {old_lens, new_lens, free_blocks, free_count};
  const fp8idx_tensor* outs[] = {bt, ctx, cu_new, slots, counts, cu_seq, ks, ke};
  for (int i = 0; i < 8; ++i) {
    if (!outs[i]) continue;
    for (const fp8idx_tensor* in : ins)
      if (tensors_overlap(in, outs[i]))
        return fail(FP8IDX_ERR_INVALID, "step tables: an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (outs[j] && tensors_overlap(outs[j], outs[i]))
        return fail(FP8IDX_ERR_INVALID, "step tables: two outputs overlap");
  }
  StepTablesParams p;
  std::memset(&p, 0, sizeof(p));
  p.old_lens = static_cast<const int32_t*>(old_lens->data);
  p.new_lens = static_cast<const int32_t*>(new_lens->data);
  p.free_blocks = static_cast<const int32_t*>(free_blocks->data);
  p.free_count = static_cast<const int32_t*>(free_count->data);
  p.block_tables = static_cast<int32_t*>(bt->data);
  p.context_lens = static_cast<int32_t*>(ctx->data);
  p.cu_new = static_cast<int32_t*>(cu_new->data);
  p.slots = static_cast<int32_t*>(slots->data);
  p.counts = static_cast<int32_t*>(counts->data);
  p.cu_seq = cu_seq ? static_cast<int32_t*>(cu_seq->data) : nullptr;
  p.ks = ks ? static_cast<int32_t*>(ks->data) : nullptr;
  p.ke = ke ? static_cast<int32_t*>(ke->data) : nullptr;
  p.bt_stride = B > 1 ? bt->stride[0] : bt->shape[1];
  p.rows = T;
  p.free_cap = free_blocks->shape[0];
  p.batch = (int32_t)B;
  p.max_blocks = (int32_t)bt->shape[1];
  p.block_size = block_size;
  DeviceInfo dev;
  TRY(device_info(&dev));
  // a thread per row (and, for small blocks, about one per block dealt)
  const int64_t ctas = (std::max<int64_t>(T, B) + kStepThreads - 1) / kStepThreads;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, dev.sms));
  cudaError_t e = launch_step_tables(p, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "step tables launch: %s", cudaGetErrorString(e));
  return ok();
}

// A cache of keys and values [num_blocks, kv_heads, page] with pages for
// `bs` tokens: its strides and size.
fp8idx_status check_kv_pages(const fp8idx_tensor* kv, int64_t bs) {
  const int64_t page = kv->shape[2];
  if (kv->shape[0] < 1 || kv->shape[1] < 1) return fail(FP8IDX_ERR_INVALID, "kv_cache: empty");
  if (kv->stride[2] != 1) return fail(FP8IDX_ERR_INVALID, "kv_cache: pages must be contiguous");
  const bool one_block = kv->shape[0] == 1, one_head = kv->shape[1] == 1;
  if ((!one_block && (kv->stride[0] % 16 != 0 || kv->stride[0] < page)) ||
      (!one_head && (kv->stride[1] % 16 != 0 || kv->stride[1] < page)))
    return fail(FP8IDX_ERR_INVALID, "kv_cache: block and head strides must be multiples of 16 bytes, at least a page");
  if (!one_block && !one_head && kv->stride[0] < kv->shape[1] * kv->stride[1] &&
      kv->stride[1] < kv->shape[0] * kv->stride[0])
    return fail(FP8IDX_ERR_INVALID, "kv_cache: the pages of blocks and heads overlap");
  if (!aligned16(kv->data)) return fail(FP8IDX_ERR_INVALID, "kv_cache must be 16-byte aligned");
  if (kv->shape[0] * bs >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "kv_cache: %lld blocks of %lld tokens (slots must stay below 2^31)",
                (long long)kv->shape[0], (long long)bs);
  return FP8IDX_OK;
}

// A key/value cache [num_blocks, kv_heads, page]: its strides, and the block
// size that its page has for head_dim D.
fp8idx_status check_kv_cache(const fp8idx_tensor* kv, int64_t D, int64_t* block_size) {
  TRY(check_tensor(kv, "kv_cache", FP8IDX_U8, 3));
  const int64_t page = kv->shape[2], bs = page / (2 * D + 8);
  if (bs < 1 || kv_page_bytes(bs, D) != page)
    return fail(FP8IDX_ERR_INVALID, "kv_cache: a page of %lld bytes is not fp8idx_kv_page_bytes(block_size, %lld)",
                (long long)page, (long long)D);
  if (!block_size_ok(bs))
    return fail(FP8IDX_ERR_UNSUPPORTED, "kv_cache: block_size %lld not in {1, 16, 32, 64, 128}", (long long)bs);
  TRY(check_kv_pages(kv, bs));
  *block_size = bs;
  return FP8IDX_OK;
}

// The same for a cache whose blocks share a scale.
fp8idx_status check_kv_block_cache(const fp8idx_tensor* kv, int64_t D, int64_t* block_size) {
  TRY(check_tensor(kv, "kv_cache", FP8IDX_U8, 3));
  const int64_t page = kv->shape[2], bs = (page - 16) / (2 * D);
  if (bs < 1 || kv_block_page_bytes(bs, D) != page)
    return fail(FP8IDX_ERR_INVALID, "kv_cache: a page of %lld bytes is not fp8idx_kv_block_page_bytes(block_size, %lld)",
                (long long)page, (long long)D);
  if (bs == 1 || !block_size_ok(bs))
    return fail(FP8IDX_ERR_UNSUPPORTED, "kv_cache: block_size %lld not in {16, 32, 64, 128}", (long long)bs);
  TRY(check_kv_pages(kv, bs));
  *block_size = bs;
  return FP8IDX_OK;
}

// The type of rows of values, or a refusal.
fp8idx_status row_type(const fp8idx_tensor* x, const char* name, int* type) {
  if (!x) return fail(FP8IDX_ERR_INVALID, "%s: null descriptor", name);
  *type = x->dtype == FP8IDX_BF16 ? kRowBf16 : x->dtype == FP8IDX_F16 ? kRowF16 : x->dtype == FP8IDX_F32 ? kRowF32 : -1;
  if (*type < 0) return fail(FP8IDX_ERR_INVALID, "%s: wrong dtype %d", name, x->dtype);
  return FP8IDX_OK;
}

// Rows [tokens, heads, D] that are read or written 16 bytes at a time: unit
// inner stride, and the byte strides of tokens and heads.
fp8idx_status check_rows(const fp8idx_tensor* x, const char* name, int64_t* token_stride, int64_t* head_stride) {
  if (x->shape[2] > 1 && x->stride[2] != 1) return fail(FP8IDX_ERR_INVALID, "%s: rows must have unit inner stride", name);
  const int64_t item = element_bytes(x->dtype);
  *token_stride = x->shape[0] > 1 ? x->stride[0] * item : 0;
  *head_stride = x->shape[1] > 1 ? x->stride[1] * item : 0;
  if (!aligned16(x->data) || *token_stride % 16 != 0 || *head_stride % 16 != 0)
    return fail(FP8IDX_ERR_INVALID, "%s: rows must be 16-byte aligned", name);
  if (*token_stride < 0 || *head_stride < 0) return fail(FP8IDX_ERR_INVALID, "%s: negative stride", name);
  return FP8IDX_OK;
}

// Whether rows of an output [tokens, heads, D] share bytes.
bool rows_overlap(const fp8idx_tensor* y) {
  for (int i = 0; i < 2; ++i)
    if (y->shape[i] > 1 && y->stride[i] < y->shape[2]) return true;
  return Extent(y).overlaps_itself();
}

// The same bytes, element for element.
bool same_view(const fp8idx_tensor* a, const fp8idx_tensor* b) {
  if (a->data != b->data) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
  return true;
}

fp8idx_status head_norm_rope_impl(const fp8idx_tensor* q, const fp8idx_tensor* k, const fp8idx_tensor* positions,
                                  const fp8idx_tensor* inv_freq, const fp8idx_tensor* q_weight,
                                  const fp8idx_tensor* q_bias, const fp8idx_tensor* k_weight,
                                  const fp8idx_tensor* k_bias, const fp8idx_norm_rope_options* opts,
                                  const fp8idx_tensor* out_q, const fp8idx_tensor* out_k, void* stream) {
  g_last_error.clear();
  const fp8idx_norm_rope_options o = opts ? *opts : fp8idx_norm_rope_options{0, 0, 0, 1e-6f, 1.f};
  int type = -1;
  TRY(row_type(q, "q", &type));
  TRY(check_tensor(q, "q", q->dtype, 3));
  const int64_t T = q->shape[0], D = q->shape[2];
  if ((k == nullptr) != (out_k == nullptr)) return fail(FP8IDX_ERR_INVALID, "k and out_k go together");
  if (!k && (k_weight || k_bias)) return fail(FP8IDX_ERR_INVALID, "k_weight or k_bias without k");
  NormRopeParams p;
  std::memset(&p, 0, sizeof(p));
  const fp8idx_tensor *xs[2] = {q, k}, *ys[2] = {out_q, out_k};
  const fp8idx_tensor *weights[2] = {q_weight, k_weight}, *biases[2] = {q_bias, k_bias};
  const char *xn[2] = {"q", "k"}, *yn[2] = {"out_q", "out_k"};
  const char *wn[2] = {"q_weight", "k_weight"}, *bn[2] = {"q_bias", "k_bias"};
  if (o.norm != kNormNone && o.norm != kNormRms && o.norm != kNormLayer)
    return fail(FP8IDX_ERR_INVALID, "norm: %d (0 none, 1 root mean square, 2 layer)", o.norm);
  if (!std::isfinite(o.eps) || o.eps < 0.f) return fail(FP8IDX_ERR_INVALID, "eps must be finite and not negative");
  if (!std::isfinite(o.rope_scale)) return fail(FP8IDX_ERR_INVALID, "rope_scale must be finite");
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    TRY(check_tensor(xs[i], xn[i], q->dtype, 3));
    TRY(check_tensor(ys[i], yn[i], q->dtype, 3));
    if (xs[i]->shape[0] != T || xs[i]->shape[2] != D) return fail(FP8IDX_ERR_INVALID, "k must have the tokens and head_dim of q");
    for (int d = 0; d < 3; ++d)
      if (ys[i]->shape[d] != xs[i]->shape[d]) return fail(FP8IDX_ERR_INVALID, "%s must have the shape of %s", yn[i], xn[i]);
    TRY(check_rows(xs[i], xn[i], &p.x_token[i], &p.x_head[i]));
    TRY(check_rows(ys[i], yn[i], &p.y_token[i], &p.y_head[i]));
    if (rows_overlap(ys[i])) return fail(FP8IDX_ERR_INVALID, "%s: rows overlap", yn[i]);
    p.x[i] = xs[i]->data;
    p.y[i] = ys[i]->data;
    p.heads[i] = (int32_t)std::min<int64_t>(xs[i]->shape[1], 1 << 30);
    const fp8idx_tensor* vs[2] = {weights[i], biases[i]};
    for (int j = 0; j < 2; ++j) {
      if (!vs[j]) continue;
      if (o.norm == kNormNone) return fail(FP8IDX_ERR_INVALID, "%s without a norm", j ? bn[i] : wn[i]);
      TRY(check_tensor(vs[j], j ? bn[i] : wn[i], FP8IDX_F32, 1));
      if (vs[j]->shape[0] != D || (D > 1 && vs[j]->stride[0] != 1))
        return fail(FP8IDX_ERR_INVALID, "%s: expected contiguous [%lld]", j ? bn[i] : wn[i], (long long)D);
      (j ? p.bias : p.weight)[i] = static_cast<const float*>(vs[j]->data);
    }
  }
  if (D < 8 || D > kNormRopeMaxDim || D % 8 != 0)
    return fail(FP8IDX_ERR_UNSUPPORTED, "head_norm_rope: head_dim %lld (a multiple of 8, 8 to %d)", (long long)D, kNormRopeMaxDim);
  TRY(check_vector(positions, "positions", T));
  TRY(check_tensor(inv_freq, "inv_freq", FP8IDX_F32, 1));
  if (inv_freq->shape[0] > 1 && inv_freq->stride[0] != 1) return fail(FP8IDX_ERR_INVALID, "inv_freq must be contiguous");
  const int64_t rot = 2 * inv_freq->shape[0], unit = o.interleaved ? 8 : 16;
  if (o.rot_start < 0 || o.rot_start + rot > D)
    return fail(FP8IDX_ERR_INVALID, "the rotated part [%d, %lld) lies outside the head", o.rot_start, (long long)(o.rot_start + rot));
  if (rot % unit != 0 || o.rot_start % 8 != 0)
    return fail(FP8IDX_ERR_UNSUPPORTED, "head_norm_rope: %lld rotated elements from %d on (multiples of %lld and 8)",
                (long long)rot, o.rot_start, (long long)unit);
  const int64_t H = q->shape[1] + (k ? k->shape[1] : 0);
  if (T >= (1ll << 31) || H >= (1ll << 31) || T * H >= (1ll << 31) - 4096)
    return fail(FP8IDX_ERR_UNSUPPORTED, "head_norm_rope: %lld tokens of %lld heads in one call", (long long)T, (long long)H);
  if (T == 0 || H == 0) return ok();
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    const fp8idx_tensor* ins[] = {q, k, positions, inv_freq, q_weight, q_bias, k_weight, k_bias};
    for (const fp8idx_tensor* in : ins)
      if (in && !(in == xs[i] && same_view(in, ys[i])) && tensors_overlap(ys[i], in))
        return fail(FP8IDX_ERR_INVALID, "%s overlaps an input (only its own rows may be the same tensor)", yn[i]);
  }
  if (k && tensors_overlap(out_q, out_k)) return fail(FP8IDX_ERR_INVALID, "out_q and out_k overlap");
  p.positions = static_cast<const int32_t*>(positions->data);
  p.inv_freq = static_cast<const float*>(inv_freq->data);
  p.tokens = (int32_t)T;
  p.dim = (int32_t)D;
  p.rot = (int32_t)rot;
  p.rot_start = o.rot_start;
  p.norm = o.norm;
  p.eps = o.eps;
  p.inv_dim = 1.f / (float)D;
  p.rope_scale = o.rope_scale;
  DeviceInfo dev;
  TRY(device_info(&dev));
  cudaError_t e = launch_norm_rope(p, type, o.interleaved != 0, dev.sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "head_norm_rope launch: %s", cudaGetErrorString(e));
  return ok();
}

fp8idx_status block_store_impl(const fp8idx_tensor* k, const fp8idx_tensor* v, const fp8idx_tensor* slots,
                               const fp8idx_tensor* kv, void* stream) {
  g_last_error.clear();
  int type = -1;
  TRY(row_type(k, "k", &type));
  BlockStoreParams p;
  std::memset(&p, 0, sizeof(p));
  const fp8idx_tensor* xs[2] = {k, v};
  const char* names[2] = {"k", "v"};
  for (int i = 0; i < 2; ++i) {
    TRY(check_tensor(xs[i], names[i], k->dtype, 3));
    for (int d = 0; d < 3; ++d)
      if (xs[i]->shape[d] != k->shape[d]) return fail(FP8IDX_ERR_INVALID, "v must have the shape of k");
    TRY(check_rows(xs[i], names[i], &p.token_stride[i], &p.head_stride[i]));
    p.x[i] = xs[i]->data;
  }
  const int64_t T = k->shape[0], H = k->shape[1], D = k->shape[2];
  TRY(check_vector(slots, "slot_mapping", T));
  if (!row_dim_ok(D)) return fail(FP8IDX_ERR_UNSUPPORTED, "block store: head_dim %lld (64 or 128)", (long long)D);
  int64_t bs = 0;
  TRY(check_kv_block_cache(kv, D, &bs));
  if (kv->shape[1] != H) return fail(FP8IDX_ERR_INVALID, "kv_cache has %lld heads, k has %lld", (long long)kv->shape[1], (long long)H);
  if (T >= (1ll << 31) || T * H >= (1ll << 30) - 4096)
    return fail(FP8IDX_ERR_UNSUPPORTED, "block store: %lld tokens of %lld heads in one call", (long long)T, (long long)H);
  if (T == 0) return ok();
  if (tensors_overlap(kv, k) || tensors_overlap(kv, v) || tensors_overlap(kv, slots))
    return fail(FP8IDX_ERR_INVALID, "block store: the cache overlaps an input");
  p.slots = static_cast<const int32_t*>(slots->data);
  p.cache = static_cast<uint8_t*>(kv->data);
  p.block_stride = kv->shape[0] > 1 ? kv->stride[0] : 0;
  p.cache_head_stride = H > 1 ? kv->stride[1] : 0;
  p.num_slots = (int32_t)(kv->shape[0] * bs);
  p.tokens = (int32_t)T;
  p.heads = (int32_t)H;
  while ((1 << p.block_shift) < bs) ++p.block_shift;
  DeviceInfo dev;
  TRY(device_info(&dev));
  cudaError_t e = launch_block_store(p, type, (int)D, dev.sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "block store launch: %s", cudaGetErrorString(e));
  return ok();
}

fp8idx_status block_attn_impl(const fp8idx_tensor* q, const fp8idx_tensor* kv, const fp8idx_tensor* bt,
                              const fp8idx_tensor* ctx, const fp8idx_tensor* cu, float softmax_scale, int32_t window,
                              const fp8idx_tensor* out, const fp8idx_tensor* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  g_last_error.clear();
  TRY(check_tensor(q, "q", FP8IDX_BF16, 3));
  TRY(check_tensor(out, "out", FP8IDX_BF16, 3));
  const int64_t R = q->shape[0], H = q->shape[1], D = q->shape[2];
  for (int i = 0; i < 3; ++i)
    if (out->shape[i] != q->shape[i]) return fail(FP8IDX_ERR_INVALID, "out must have the shape of q");
  if (!row_dim_ok(D)) return fail(FP8IDX_ERR_UNSUPPORTED, "block attention: head_dim %lld (64 or 128)", (long long)D);
  int64_t q_token, q_head, out_token, out_head;
  TRY(check_rows(q, "q", &q_token, &q_head));
  TRY(check_rows(out, "out", &out_token, &out_head));
  if (H < 1) return fail(FP8IDX_ERR_INVALID, "q has no heads");
  if (rows_overlap(out)) return fail(FP8IDX_ERR_INVALID, "out: rows overlap");
  int64_t bs = 0;
  TRY(check_kv_block_cache(kv, D, &bs));
  const int64_t HK = kv->shape[1];
  if (H % HK != 0) return fail(FP8IDX_ERR_INVALID, "%lld heads are no multiple of %lld kv_heads", (long long)H, (long long)HK);
  if (H / HK > kBlockAttnMaxGroup)
    return fail(FP8IDX_ERR_UNSUPPORTED, "block attention: %lld heads per key head (at most %d)", (long long)(H / HK), kBlockAttnMaxGroup);
  TRY(check_tensor(bt, "block_tables", FP8IDX_I32, 2));
  const int64_t B = bt->shape[0];
  if (bt->shape[1] > 1 && bt->stride[1] != 1) return fail(FP8IDX_ERR_INVALID, "block_tables rows must be contiguous");
  if (B > 1 && bt->stride[0] < 0) return fail(FP8IDX_ERR_INVALID, "block_tables: negative stride");
  if (B > kMaxBatch) return fail(FP8IDX_ERR_UNSUPPORTED, "block attention: %lld requests > %d", (long long)B, kMaxBatch);
  if (bt->shape[1] * bs >= (1ll << 31) - 256) return fail(FP8IDX_ERR_UNSUPPORTED, "positions must stay below 2^31 - 256");
  TRY(check_vector(ctx, "context_lens", B));
  TRY(check_vector(cu, "cu_new_lens", B + 1));
  if (window < 0) return fail(FP8IDX_ERR_INVALID, "window must not be negative (0: every position up to the row's own)");
  if (lse) {
    TRY(check_tensor(lse, "lse", FP8IDX_F32, 2));
    if (lse->shape[0] != R || lse->shape[1] != H || !contiguous(lse))
      return fail(FP8IDX_ERR_INVALID, "lse must be contiguous [rows, heads]");
  }
  if (!std::isfinite(softmax_scale * 1.4426950408889634f)) return fail(FP8IDX_ERR_INVALID, "softmax_scale must be finite (times log2 e, too)");
  if (R >= (1ll << 31) || R * H >= (1ll << 31) - 4096) return fail(FP8IDX_ERR_UNSUPPORTED, "block attention: rows*heads must stay below 2^31");
  const size_t need = block_attn_workspace((int)D);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return fail(FP8IDX_ERR_INVALID, "workspace must be 256-byte aligned device memory");
  if (workspace_bytes < need)
    return fail(FP8IDX_ERR_INVALID, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (R == 0 || B == 0) return ok();
  if (bt->shape[1] < 1) return fail(FP8IDX_ERR_INVALID, "empty block table");
  const fp8idx_tensor ws{workspace, FP8IDX_U8, 1, {(int64_t)need, 0, 0, 0}, {1, 0, 0, 0}};
  const fp8idx_tensor* ins[] = {q, kv, bt, ctx, cu};
  for (const fp8idx_tensor* in : ins)
    if (tensors_overlap(out, in) || (lse && tensors_overlap(lse, in)) || tensors_overlap(&ws, in))
      return fail(FP8IDX_ERR_INVALID, "block attention: an output or the workspace overlaps an input");
  if ((lse && (tensors_overlap(out, lse) || tensors_overlap(&ws, lse))) || tensors_overlap(&ws, out))
    return fail(FP8IDX_ERR_INVALID, "block attention: out, lse and workspace overlap");
  BlockAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q->data;
  p.out = out->data;
  p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  p.kv = static_cast<const uint8_t*>(kv->data);
  p.block_tables = static_cast<const int32_t*>(bt->data);
  p.context_lens = static_cast<const int32_t*>(ctx->data);
  p.cu_new = static_cast<const int32_t*>(cu->data);
  p.block_stride = kv->shape[0] > 1 ? kv->stride[0] : 0;
  p.head_stride = HK > 1 ? kv->stride[1] : 0;
  p.q_row_stride = q_token / 2;
  p.q_head_stride = q_head / 2;
  p.out_row_stride = out_token / 2;
  p.out_head_stride = out_head / 2;
  p.bt_stride = B > 1 ? bt->stride[0] : 0;
  p.rows = (int32_t)R;
  p.heads = (int32_t)H;
  p.kv_heads = (int32_t)HK;
  p.group = (int32_t)(H / HK);
  while ((1 << p.block_shift) < bs) ++p.block_shift;
  p.max_blocks = (int32_t)bt->shape[1];
  p.num_blocks = (int32_t)kv->shape[0];
  p.n_req = (int32_t)B;
  p.half_positions = kBlockAttnLanes / 2 / p.group;
  p.window = window;
  p.negative = softmax_scale < 0.f;
  p.scale_log2 = (float)(std::fabs((double)softmax_scale) * 1.4426950408889634);
  p.partial = static_cast<float*>(workspace);
  p.meta = reinterpret_cast<BlockAttnMeta*>(p.partial + 2ll * kBlockAttnMaxCtas * block_attn_piece_floats((int)D));
  DeviceInfo dev;
  TRY(device_info(&dev));
  if (block_attn_smem((int)D) > dev.smem_optin)
    return fail(FP8IDX_ERR_UNSUPPORTED, "block attention: shared memory too small");
  const int64_t page = kv->shape[2];
  const uint64_t dims[4] = {(uint64_t)(2 * D), (uint64_t)bs, (uint64_t)HK, (uint64_t)kv->shape[0]};
  const uint64_t strides[3] = {(uint64_t)(2 * D), (uint64_t)(HK > 1 ? kv->stride[1] : page),
                               (uint64_t)(kv->shape[0] > 1 ? kv->stride[0] : HK * page)};
  const uint32_t box[4] = {128u, (uint32_t)bs, 1u, 1u};
  if (strides[1] >= 1ull << 40 || strides[2] >= 1ull << 40)
    return fail(FP8IDX_ERR_UNSUPPORTED, "kv_cache: strides of 2^40 bytes or more");
  CUtensorMap tm;
  TRY(encode(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, kv->data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, "kv_cache"));
  // One CTA an SM, as far as the call can have steps (of 128 positions at least) for them.
  const int64_t units = (R / (2 * p.half_positions) + B) * HK, steps = (bt->shape[1] * bs + kTileTokens - 1) / kTileTokens;
  const int grid = (int)std::min<int64_t>(std::min(dev.sms, kBlockAttnMaxCtas), units * steps);
  cudaError_t e = launch_block_attn(tm, p, (int)D, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "block attention launch: %s", cudaGetErrorString(e));
  return ok();
}

fp8idx_status paged_store_impl(const fp8idx_tensor* k, const fp8idx_tensor* v, const fp8idx_tensor* slots,
                               const fp8idx_tensor* kv, void* stream) {
  g_last_error.clear();
  const int nd = v ? 3 : 2;
  if (!k) return fail(FP8IDX_ERR_INVALID, "k: null descriptor");
  int type = -1;
  if (k->dtype == FP8IDX_BF16) type = kRowBf16;
  if (k->dtype == FP8IDX_F16) type = kRowF16;
  if (k->dtype == FP8IDX_F32) type = kRowF32;
  if (type < 0) return fail(FP8IDX_ERR_INVALID, "k: wrong dtype %d", k->dtype);
  const int64_t item = type == kRowF32 ? 4 : 2;
  TRY(check_tensor(k, "k", k->dtype, nd));
  const int64_t T = k->shape[0], H = v ? k->shape[1] : 1, D = k->shape[nd - 1];
  PagedStoreParams p;
  std::memset(&p, 0, sizeof(p));
  const fp8idx_tensor* xs[2] = {k, v};
  for (int i = 0; i < (v ? 2 : 1); ++i) {
    const fp8idx_tensor* x = xs[i];
    const char* name = i ? "v" : "k";
    TRY(check_tensor(x, name, k->dtype, nd));
    for (int d = 0; d < nd; ++d)
      if (x->shape[d] != k->shape[d]) return fail(FP8IDX_ERR_INVALID, "v must have the shape of k");
    if (x->stride[nd - 1] != 1) return fail(FP8IDX_ERR_INVALID, "%s: rows must have unit inner stride", name);
    p.x[i] = x->data;
    p.token_stride[i] = T > 1 ? x->stride[0] * item : 0;
    p.head_stride[i] = v && H > 1 ? x->stride[1] * item : 0;
    if (!aligned16(x->data) || p.token_stride[i] % 16 != 0 || p.head_stride[i] % 16 != 0)
      return fail(FP8IDX_ERR_INVALID, "%s: rows must be 16-byte aligned", name);
  }
  TRY(check_vector(slots, "slot_mapping", T));
  if (!row_dim_ok(D)) return fail(FP8IDX_ERR_UNSUPPORTED, "store: head_dim %lld (64 or 128)", (long long)D);
  int64_t bs = 0;
  if (v) {
    TRY(check_kv_cache(kv, D, &bs));
    if (kv->shape[1] != H) return fail(FP8IDX_ERR_INVALID, "kv_cache has %lld heads, k has %lld", (long long)kv->shape[1], (long long)H);
    p.block_stride = kv->shape[0] > 1 ? kv->stride[0] : 0;
    p.cache_head_stride = H > 1 ? kv->stride[1] : 0;
  } else {
    TRY(check_tensor(kv, "kv_cache", FP8IDX_U8, 2));
    if (!contiguous(kv)) return fail(FP8IDX_ERR_INVALID, "kv_cache must be contiguous");
    if (kv->shape[0] < 1 || kv->shape[1] < 1 || kv->shape[1] % (D + 4) != 0)
      return fail(FP8IDX_ERR_INVALID, "kv_cache rows must be block_size*(head_dim+4) bytes");
    bs = kv->shape[1] / (D + 4);
    if (!block_size_ok(bs))
      return fail(FP8IDX_ERR_UNSUPPORTED, "store: block_size %lld not in {1, 16, 32, 64, 128}", (long long)bs);
    if (!aligned16(kv->data)) return fail(FP8IDX_ERR_INVALID, "kv_cache must be 16-byte aligned");
    if (kv->shape[0] * bs >= (1ll << 31)) return fail(FP8IDX_ERR_UNSUPPORTED, "store: slots must stay below 2^31");
    p.block_stride = kv->shape[1];
  }
  if (T * H * (v ? 2 : 1) >= (1ll << 31) - 4096)
    return fail(FP8IDX_ERR_UNSUPPORTED, "store: %lld tokens of %lld heads in one call", (long long)T, (long long)H);
  if (T == 0 || H == 0) return ok();
  if (tensors_overlap(kv, k) || (v && tensors_overlap(kv, v)) || tensors_overlap(kv, slots))
    return fail(FP8IDX_ERR_INVALID, "store: the cache overlaps an input");
  p.slots = static_cast<const int32_t*>(slots->data);
  p.cache = static_cast<uint8_t*>(kv->data);
  p.num_slots = kv->shape[0] * bs;
  p.tokens = T;
  p.heads = (int32_t)H;
  while ((1 << p.block_shift) < bs) ++p.block_shift;
  // rows are numbered below 2^31: with s = ceil(log2 d), row / d is
  // row * ceil(2^(31+s) / d) >> (31 + s)
  const uint64_t d = (uint64_t)H * (v ? 2 : 1);
  p.div_shift = -1;
  if (d > 1) {
    int s = 1;
    while ((1ull << s) < d) ++s;
    p.div_mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
    p.div_shift = s - 1;
  }
  DeviceInfo dev;
  TRY(device_info(&dev));
  cudaError_t e = launch_paged_store(p, type, (int)D, dev.sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "store launch: %s", cudaGetErrorString(e));
  return ok();
}

// decode: q [batch, next_n, heads, D], cu_seq null; prefill: q [M, heads, D].
fp8idx_status sparse_attn_impl(const fp8idx_tensor* q, const fp8idx_tensor* kv, const fp8idx_tensor* bt,
                               const fp8idx_tensor* cu, bool prefill, const fp8idx_tensor* idx, float softmax_scale,
                               const fp8idx_tensor* out, const fp8idx_tensor* lse, const fp8idx_options* opts,
                               void* stream) {
  g_last_error.clear();
  const int nd = prefill ? 3 : 4;
  TRY(check_tensor(q, "q", FP8IDX_BF16, nd));
  TRY(check_tensor(out, "out", FP8IDX_BF16, nd));
  const int64_t H = q->shape[nd - 2], D = q->shape[nd - 1];
  const int64_t n = prefill ? 1 : q->shape[1], B = q->shape[0], R = B * n;
  for (int i = 0; i < nd; ++i)
    if (out->shape[i] != q->shape[i]) return fail(FP8IDX_ERR_INVALID, "out must have the shape of q");
  if (!row_dim_ok(D)) return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: head_dim %lld (64 or 128)", (long long)D);
  if (q->stride[nd - 1] != 1 || out->stride[nd - 1] != 1)
    return fail(FP8IDX_ERR_INVALID, "q and out must have unit inner stride");
  for (int i = 0; i < nd - 1; ++i) {
    if (q->shape[i] > 1 && q->stride[i] < 0) return fail(FP8IDX_ERR_INVALID, "q: negative stride");
    if (out->shape[i] > 1 && out->stride[i] < D) return fail(FP8IDX_ERR_INVALID, "out: rows overlap");
  }
  if (Extent(out).overlaps_itself()) return fail(FP8IDX_ERR_INVALID, "out: rows overlap");
  if (H < 1 || n < 1) return fail(FP8IDX_ERR_INVALID, "q has no heads or rows per request");
  int64_t bs = 0;
  TRY(check_kv_cache(kv, D, &bs));
  const int64_t HK = kv->shape[1];
  if (H % HK != 0) return fail(FP8IDX_ERR_INVALID, "%lld heads are no multiple of %lld kv_heads", (long long)H, (long long)HK);
  if (H / HK > kAttnMaxGroup)
    return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: %lld heads per key head (at most %d)", (long long)(H / HK), kAttnMaxGroup);
  TRY(check_tensor(bt, "block_tables", FP8IDX_I32, 2));
  if (bt->shape[1] > 1 && bt->stride[1] != 1) return fail(FP8IDX_ERR_INVALID, "block_tables rows must be contiguous");
  if (!prefill && bt->shape[0] != B) return fail(FP8IDX_ERR_INVALID, "block_tables must be [batch, max_blocks]");
  if (R > 0 && (bt->shape[1] < 1 || (prefill && bt->shape[0] < 1))) return fail(FP8IDX_ERR_INVALID, "empty block table");
  if (bt->shape[1] * bs >= (1ll << 31)) return fail(FP8IDX_ERR_UNSUPPORTED, "positions must stay below 2^31");
  if (prefill) {
    if (bt->shape[0] > kMaxBatch)
      return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: %lld requests > %d", (long long)bt->shape[0], kMaxBatch);
    TRY(check_vector(cu, "cu_seq_lens", bt->shape[0] + 1));
  }
  TRY(check_tensor(idx, "indices", FP8IDX_I32, 2));
  const int64_t k = idx->shape[1];
  if (k < 1 || k > kAttnMaxK) return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: k=%lld not in [1, %d]", (long long)k, kAttnMaxK);
  if (idx->shape[0] != R || (k > 1 && idx->stride[1] != 1) || (R > 1 && idx->stride[0] < 0))
    return fail(FP8IDX_ERR_INVALID, "indices must be [rows, k] with unit inner stride");
  if (lse) {
    TRY(check_tensor(lse, "lse", FP8IDX_F32, 2));
    if (lse->shape[0] != R || lse->shape[1] != H || !contiguous(lse))
      return fail(FP8IDX_ERR_INVALID, "lse must be contiguous [rows, heads]");
  }
  if (!std::isfinite(softmax_scale * 1.4426950408889634f)) return fail(FP8IDX_ERR_INVALID, "softmax_scale must be finite (times log2 e, too)");
  if (R * H >= (1ll << 31)) return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: rows*heads must stay below 2^31");
  const int32_t ctas = opts ? opts->num_ctas : 0;
  if (ctas != 0 && ctas != 1 && ctas != 2 && ctas != 4 && ctas != 8)
    return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: num_ctas=%d not in {0, 1, 2, 4, 8}", ctas);
  if (R == 0) return ok();
  SparseAttnParams p;
  std::memset(&p, 0, sizeof(p));
  const auto strides = [&](const fp8idx_tensor* t, int64_t* req, int64_t* row, int64_t* head) {
    *req = B > 1 ? t->stride[0] : 0;
    *row = !prefill && n > 1 ? t->stride[1] : 0;
    *head = H > 1 ? t->stride[nd - 2] : 0;
  };
  strides(q, &p.q_req_stride, &p.q_row_stride, &p.q_head_stride);
  strides(out, &p.out_req_stride, &p.out_row_stride, &p.out_head_stride);
  if (!aligned16(q->data) || ((p.q_req_stride | p.q_row_stride | p.q_head_stride) & 7) != 0)
    return fail(FP8IDX_ERR_INVALID, "q rows must be 16-byte aligned");
  p.q = q->data;
  p.out = out->data;
  p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  p.kv = static_cast<const uint8_t*>(kv->data);
  p.indices = static_cast<const int32_t*>(idx->data);
  p.block_tables = static_cast<const int32_t*>(bt->data);
  p.cu_seq_lens = prefill ? static_cast<const int32_t*>(cu->data) : nullptr;
  p.idx_stride = R > 1 ? idx->stride[0] : k;
  const int64_t bt_stride = bt->shape[0] > 1 ? bt->stride[0] : 0;
  if (bt_stride < 0 || bt_stride >= (1ll << 31)) return fail(FP8IDX_ERR_UNSUPPORTED, "block_tables: row stride of 2^31 or more");
  p.bt_stride = (int32_t)bt_stride;
  const int64_t block_stride = kv->shape[0] > 1 ? kv->stride[0] : 0, head_stride = HK > 1 ? kv->stride[1] : 0;
  int64_t unit = 16;
  while (((block_stride | head_stride | 2 * D) & (2 * unit - 1)) == 0) unit *= 2;
  if ((kv->shape[0] - 1) * block_stride + (HK - 1) * head_stride + kv->shape[2] >= unit << 32)
    return fail(FP8IDX_ERR_UNSUPPORTED, "kv_cache: spans %lld bytes or more (offsets are 2^32 multiples of %lld)",
                (long long)(unit << 32), (long long)unit);
  p.unit = (uint32_t)unit;
  p.block_units = (uint32_t)(block_stride / unit);
  p.head_units = (uint32_t)(head_stride / unit);
  p.tok_units = (uint32_t)(2 * D / unit);
  p.scale_off = (int32_t)(bs * 2 * D);
  p.num_blocks = (int32_t)kv->shape[0];
  p.heads = (int32_t)H;
  p.kv_heads = (int32_t)HK;
  p.group = (int32_t)(H / HK);
  p.next_n = (int32_t)n;
  p.k = (int32_t)k;
  p.max_blocks = (int32_t)bt->shape[1];
  p.block_size = (int32_t)bs;
  p.n_req = (int32_t)bt->shape[0];
  p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  while ((1 << p.block_shift) < p.block_size) ++p.block_shift;
  const int gp = attn_pad(p.group);
  p.head_chunks = (p.group + gp - 1) / gp;
  if (R * HK * p.head_chunks * kAttnMaxCtas >= (1ll << 31))
    return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: too many rows");
  p.units = (int32_t)(R * HK * p.head_chunks);
  p.tiles = (int32_t)((k + kAttnTile - 1) / kAttnTile);
  const fp8idx_tensor* ins[] = {q, kv, idx, bt, prefill ? cu : bt};
  for (const fp8idx_tensor* in : ins)
    if (tensors_overlap(out, in) || (lse && tensors_overlap(lse, in)))
      return fail(FP8IDX_ERR_INVALID, "sparse attention: an output overlaps an input");
  if (lse && tensors_overlap(out, lse)) return fail(FP8IDX_ERR_INVALID, "sparse attention: out and lse overlap");
  DeviceInfo dev;
  TRY(device_info(&dev));
  // Persistent CTAs (two units at a time), or a cluster of CTAs per unit
  // (which share its tiles): whichever leaves the busiest SM the least to do,
  // in tiles, a cluster's start, meeting and end counted as about six.
  int cs = ctas;
  if (ctas == 0) {
    const int64_t pair = static_cast<int64_t>(kAttnGroups) * dev.sms;
    int64_t best = (p.units + pair - 1) / pair * kAttnGroups * p.tiles + 2;
    for (int c = 1; c <= kAttnMaxCtas && (c == 1 || c / 2 < p.tiles); c *= 2) {
      const int64_t waves = (static_cast<int64_t>(p.units) * c + dev.sms - 1) / dev.sms;
      const int64_t cost = waves * ((p.tiles + c - 1) / c + 6);
      if (cost < best) cs = c, best = cost;
    }
  }
  const int grid = cs == 0 ? std::min(p.units, dev.sms) : p.units * cs;
  const int smem = (int)attn_smem_layout((int)D, gp).total;
  if (smem > dev.smem_optin) return fail(FP8IDX_ERR_UNSUPPORTED, "sparse attention: shared memory too small");
  cudaError_t e = launch_sparse_attn(p, (int)D, grid, cs, smem, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "sparse attention launch: %s", cudaGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

fp8idx_status fp8_paged_mqa_logits(const fp8idx_tensor* q_fp8, const fp8idx_tensor* kv_cache,
                                   const fp8idx_tensor* weights, const fp8idx_tensor* context_lens,
                                   const fp8idx_tensor* block_tables, int32_t max_model_len,
                                   const fp8idx_tensor* out, void* stream) {
  return paged_impl(q_fp8, kv_cache, weights, context_lens, block_tables, max_model_len, out, nullptr, stream);
}

fp8idx_status fp8_paged_mqa_logits_ex(const fp8idx_tensor* q_fp8, const fp8idx_tensor* kv_cache,
                                      const fp8idx_tensor* weights, const fp8idx_tensor* context_lens,
                                      const fp8idx_tensor* block_tables, int32_t max_model_len,
                                      const fp8idx_tensor* out, const fp8idx_options* opts, void* stream) {
  return paged_impl(q_fp8, kv_cache, weights, context_lens, block_tables, max_model_len, out, opts, stream);
}

fp8idx_status fp8_mqa_logits(const fp8idx_tensor* q_fp8, const fp8idx_tensor* k_fp8, const fp8idx_tensor* kv_scale,
                             const fp8idx_tensor* weights, const fp8idx_tensor* cu_seqlen_ks,
                             const fp8idx_tensor* cu_seqlen_ke, const fp8idx_tensor* out, void* stream) {
  PrefillK src;
  src.k = k_fp8;
  src.s = kv_scale;
  return prefill_impl(q_fp8, src, weights, cu_seqlen_ks, cu_seqlen_ke, out, nullptr, stream);
}

fp8idx_status fp8_mqa_logits_ex(const fp8idx_tensor* q_fp8, const fp8idx_tensor* k_fp8,
                                const fp8idx_tensor* kv_scale, const fp8idx_tensor* weights,
                                const fp8idx_tensor* cu_seqlen_ks, const fp8idx_tensor* cu_seqlen_ke,
                                const fp8idx_tensor* out, const fp8idx_options* opts, void* stream) {
  PrefillK src;
  src.k = k_fp8;
  src.s = kv_scale;
  return prefill_impl(q_fp8, src, weights, cu_seqlen_ks, cu_seqlen_ke, out, opts, stream);
}

fp8idx_status fp8_mqa_logits_paged(const fp8idx_tensor* q_fp8, const fp8idx_tensor* kv_cache,
                                   const fp8idx_tensor* block_tables, const fp8idx_tensor* cu_seq_lens,
                                   const fp8idx_tensor* weights, const fp8idx_tensor* cu_seqlen_ks,
                                   const fp8idx_tensor* cu_seqlen_ke, const fp8idx_tensor* out,
                                   const fp8idx_options* opts, void* stream) {
  PrefillK src;
  src.kv = kv_cache;
  src.bt = block_tables;
  src.cu = cu_seq_lens;
  return prefill_impl(q_fp8, src, weights, cu_seqlen_ks, cu_seqlen_ke, out, opts, stream);
}

fp8idx_status fp8_paged_mqa_topk(const fp8idx_tensor* q_fp8, const fp8idx_tensor* kv_cache,
                                 const fp8idx_tensor* weights, const fp8idx_tensor* context_lens,
                                 const fp8idx_tensor* block_tables, int32_t max_model_len, int32_t k,
                                 const fp8idx_tensor* indices, void* workspace, size_t workspace_bytes,
                                 const fp8idx_options* opts, void* stream) {
  return paged_topk_impl(q_fp8, kv_cache, weights, context_lens, block_tables, max_model_len, k, indices, workspace,
                         workspace_bytes, opts, stream);
}

size_t fp8idx_paged_mqa_topk_workspace(int64_t batch, int32_t next_n, int32_t max_model_len, int32_t k) {
  if (batch < 0 || next_n < 1 || max_model_len < 0 || k < 1 || k > kTopkMaxK) return 0;
  return paged_topk_workspace(batch, next_n, max_model_len, k);
}

fp8idx_status fp8_paged_topk(const fp8idx_tensor* logits, const fp8idx_tensor* context_lens, int32_t next_n,
                             int32_t max_model_len, int32_t k, const fp8idx_tensor* indices, void* stream) {
  return topk_impl(1, logits, nullptr, nullptr, context_lens, next_n, max_model_len, k, indices, nullptr, stream);
}

fp8idx_status fp8_mqa_topk(const fp8idx_tensor* logits, const fp8idx_tensor* cu_seqlen_ks,
                           const fp8idx_tensor* cu_seqlen_ke, int32_t k, const fp8idx_tensor* indices, void* stream) {
  return topk_impl(0, logits, cu_seqlen_ks, cu_seqlen_ke, nullptr, 1, 0, k, indices, nullptr, stream);
}
fp8idx_status fp8_paged_topk_ex(const fp8idx_tensor* logits, const fp8idx_tensor* context_lens, int32_t next_n,
                                int32_t max_model_len, int32_t k, const fp8idx_tensor* indices,
                                const fp8idx_options* opts, void* stream) {
  return topk_impl(1, logits, nullptr, nullptr, context_lens, next_n, max_model_len, k, indices, opts, stream);
}
fp8idx_status fp8_mqa_topk_ex(const fp8idx_tensor* logits, const fp8idx_tensor* cu_seqlen_ks,
                              const fp8idx_tensor* cu_seqlen_ke, int32_t k, const fp8idx_tensor* indices,
                              const fp8idx_options* opts, void* stream) {
  return topk_impl(0, logits, cu_seqlen_ks, cu_seqlen_ke, nullptr, 1, 0, k, indices, opts, stream);
}

int64_t fp8idx_kv_page_bytes(int32_t block_size, int32_t head_dim) {
  return block_size_ok(block_size) && row_dim_ok(head_dim) ? kv_page_bytes(block_size, head_dim) : 0;
}

fp8idx_status fp8idx_paged_step_tables(const fp8idx_tensor* old_lens, const fp8idx_tensor* new_lens,
                                       const fp8idx_tensor* free_blocks, const fp8idx_tensor* free_count,
                                       int32_t block_size, const fp8idx_tensor* block_tables,
                                       const fp8idx_tensor* context_lens, const fp8idx_tensor* cu_new_lens,
                                       const fp8idx_tensor* slot_mapping, const fp8idx_tensor* counts,
                                       const fp8idx_tensor* cu_seq_lens, const fp8idx_tensor* cu_seqlen_ks,
                                       const fp8idx_tensor* cu_seqlen_ke, void* stream) {
  return step_tables_impl(old_lens, new_lens, free_blocks, free_count, block_size, block_tables, context_lens,
                          cu_new_lens, slot_mapping, counts, cu_seq_lens, cu_seqlen_ks, cu_seqlen_ke, stream);
}

fp8idx_status fp8_paged_store(const fp8idx_tensor* k, const fp8idx_tensor* v, const fp8idx_tensor* slot_mapping,
                              const fp8idx_tensor* kv_cache, void* stream) {
  return paged_store_impl(k, v, slot_mapping, kv_cache, stream);
}

int64_t fp8idx_kv_block_page_bytes(int32_t block_size, int32_t head_dim) {
  return block_size > 1 && block_size_ok(block_size) && row_dim_ok(head_dim) ? kv_block_page_bytes(block_size, head_dim) : 0;
}

fp8idx_status fp8idx_head_norm_rope(const fp8idx_tensor* q, const fp8idx_tensor* k, const fp8idx_tensor* positions,
                                    const fp8idx_tensor* inv_freq, const fp8idx_tensor* q_weight,
                                    const fp8idx_tensor* q_bias, const fp8idx_tensor* k_weight,
                                    const fp8idx_tensor* k_bias, const fp8idx_norm_rope_options* opts,
                                    const fp8idx_tensor* out_q, const fp8idx_tensor* out_k, void* stream) {
  return head_norm_rope_impl(q, k, positions, inv_freq, q_weight, q_bias, k_weight, k_bias, opts, out_q, out_k, stream);
}

fp8idx_status fp8_paged_block_store(const fp8idx_tensor* k, const fp8idx_tensor* v, const fp8idx_tensor* slot_mapping,
                                    const fp8idx_tensor* kv_cache, void* stream) {
  return block_store_impl(k, v, slot_mapping, kv_cache, stream);
}

size_t fp8idx_paged_block_attn_workspace(int32_t head_dim) {
  return row_dim_ok(head_dim) ? block_attn_workspace(head_dim) : 0;
}

fp8idx_status fp8_paged_block_attn(const fp8idx_tensor* q, const fp8idx_tensor* kv_cache,
                                   const fp8idx_tensor* block_tables, const fp8idx_tensor* context_lens,
                                   const fp8idx_tensor* cu_new_lens, float softmax_scale, int32_t window,
                                   const fp8idx_tensor* out, const fp8idx_tensor* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return block_attn_impl(q, kv_cache, block_tables, context_lens, cu_new_lens, softmax_scale, window, out, lse,
                         workspace, workspace_bytes, stream);
}

fp8idx_status fp8_paged_sparse_attn(const fp8idx_tensor* q, const fp8idx_tensor* kv_cache,
                                    const fp8idx_tensor* indices, const fp8idx_tensor* block_tables,
                                    float softmax_scale, const fp8idx_tensor* out, const fp8idx_tensor* lse,
                                    const fp8idx_options* opts, void* stream) {
  return sparse_attn_impl(q, kv_cache, block_tables, nullptr, false, indices, softmax_scale, out, lse, opts, stream);
}

fp8idx_status fp8_mqa_sparse_attn_paged(const fp8idx_tensor* q, const fp8idx_tensor* kv_cache,
                                        const fp8idx_tensor* block_tables, const fp8idx_tensor* cu_seq_lens,
                                        const fp8idx_tensor* indices, float softmax_scale, const fp8idx_tensor* out,
                                        const fp8idx_tensor* lse, const fp8idx_options* opts, void* stream) {
  return sparse_attn_impl(q, kv_cache, block_tables, cu_seq_lens, true, indices, softmax_scale, out, lse, opts, stream);
}

int fp8idx_paged_is_supported(int32_t heads, int32_t head_dim, int32_t block_size, int32_t next_n) {
  return paged_supported(heads, head_dim, block_size, next_n) ? 1 : 0;
}

int fp8idx_prefill_is_supported(int32_t heads, int32_t head_dim) { return prefill_supported(heads, head_dim) ? 1 : 0; }

int fp8idx_is_supported(int32_t heads, int32_t head_dim, int32_t kv_block_size, int32_t next_n) {
  return paged_supported(heads, head_dim, kv_block_size, next_n) ? 1 : 0;
}

fp8idx_status fp8idx_plan_paged(int32_t batch, int32_t next_n, int32_t heads, int32_t head_dim, int32_t block_size,
                                int32_t max_model_len, int32_t num_sms, const fp8idx_options* opts,
                                fp8idx_plan* plan) {
  g_last_error.clear();
  if (!plan) return fail(FP8IDX_ERR_INVALID, "plan: null output");
  int smem = kMaxSmem;
  if (num_sms <= 0) {
    DeviceInfo dev;
    TRY(device_info(&dev));
    num_sms = dev.sms;
    smem = dev.smem_optin;
  }
  return plan_paged(batch, next_n, heads, head_dim, block_size, max_model_len, num_sms, smem, opts, plan);
}

fp8idx_status fp8idx_plan_prefill(int64_t rows, int64_t cols, int32_t heads, int32_t head_dim, int32_t num_sms,
                                  const fp8idx_options* opts, fp8idx_plan* plan) {
  g_last_error.clear();
  if (!plan) return fail(FP8IDX_ERR_INVALID, "plan: null output");
  int smem = kMaxSmem;
  if (num_sms <= 0) {
    DeviceInfo dev;
    TRY(device_info(&dev));
    num_sms = dev.sms;
    smem = dev.smem_optin;
  }
  return plan_prefill(rows, cols, heads, head_dim, num_sms, smem, opts, plan);
}

const char* fp8idx_last_error(void) { return g_last_error.c_str(); }

fp8idx_status fp8idx_host_mapped_pointer(const void* host_ptr, void** device_ptr) {
  g_last_error.clear();
  if (host_ptr == nullptr || device_ptr == nullptr) return fail(FP8IDX_ERR_INVALID, "host_mapped_pointer: null argument");
  cudaPointerAttributes a;
  std::memset(&a, 0, sizeof(a));
  const cudaError_t e = cudaPointerGetAttributes(&a, host_ptr);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(FP8IDX_ERR_INVALID, "host_mapped_pointer: %s", cudaGetErrorString(e));
  }
  if (a.type != cudaMemoryTypeHost) return fail(FP8IDX_ERR_INVALID, "host_mapped_pointer: not page-locked host memory");
  if (a.devicePointer == nullptr)
    return fail(FP8IDX_ERR_UNSUPPORTED, "host_mapped_pointer: the memory is not mapped into the device");
  *device_ptr = a.devicePointer;
  return ok();
}

fp8idx_status fp8idx_device_status(int32_t clear) {
  g_last_error.clear();
  unsigned int a = 0, b = 0, c = 0, d = 0, e = 0;
  if (read_paged_watchdog(&a, clear != 0) != cudaSuccess || read_prefill_watchdog(&b, clear != 0) != cudaSuccess ||
      read_topk_watchdog(&c, clear != 0) != cudaSuccess || read_attn_watchdog(&d, clear != 0) != cudaSuccess ||
      read_block_attn_watchdog(&e, clear != 0) != cudaSuccess)
    return fail(FP8IDX_ERR_CUDA, "reading the device watchdog failed");
  if (a | b | c | d | e)
    return fail(FP8IDX_ERR_TIMEOUT,
                "device wait timed out (decode sites 0x%x, prefill sites 0x%x, top-k sites 0x%x, attention sites 0x%x, "
                "block attention sites 0x%x)",
                a, b, c, d, e);
  return FP8IDX_OK;
}

fp8idx_status fp8idx_watchdog_selftest(int32_t limit_us, void* stream) {
  g_last_error.clear();
  if (limit_us < 1 || limit_us > 100000) return fail(FP8IDX_ERR_INVALID, "limit_us %d not in [1, 100000]", limit_us);
  DeviceInfo dev;
  TRY(device_info(&dev));
  cudaError_t e = launch_watchdog_selftest(static_cast<uint64_t>(limit_us) * 1000ull, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FP8IDX_ERR_CUDA, "watchdog self-test launch: %s", cudaGetErrorString(e));
  return ok();
}

int32_t fp8idx_version(void) { return 103; }

}  // extern "C"
