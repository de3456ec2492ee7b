// Attention over the selected positions of a paged e4m3 key/value cache
// (fp8_paged_sparse_attn, fp8_mqa_sparse_attn_paged) for sm_103a.
//
//   s[h, j] = softmax_scale * <q[h], K[i_j]>,  out[h] = sum_j softmax(s)[h, j] V[i_j]
//
// A unit of work is (row, key head, up to 32 of its query heads); its entries
// are taken in tiles of 128 tokens.  Both products of a tile run on the fp8
// tensor cores straight from the cache's bytes:
//   S^T [128 tokens x 2 GP] = K tile (A, K-major) * [Qh; Ql]^T
//   O^T [128 channels x 2 GP] += V tile^T (A, MN-major) * [Ph | Pl] (B, MN-major)
// GP is the head count padded to 16 or 32.  The 16-bit operands are split
// into two e4m3 values: x = h + l / 16 with h = e4m3(x), l = e4m3(16 (x - h)).
// That keeps 8 significant bits: a bf16 query exactly (down to 2^-10 of its
// head's largest element; powers of two bring a unit, and where they are far
// apart its heads, into the range), the product of a probability and its
// value's scale to 2^-8 of itself, or to half a step of 2^-18 of the row's
// largest one.  The two halves have their own accumulator columns and meet in
// f32.  Dequantising the tile to 16 bits instead would take a conversion per
// cache byte and twice the shared memory.
//
// A CTA (20 warps) is two pipelines side by side, which share nothing but two
// warps that split the next unit's query.  Each has
//  * four producer warps: a lane resolves one entry of the tile to its cache
//    row (indices are loaded two tiles ahead, block-table entries one), then
//    the warp copies its 32 rows, 16 bytes a lane, into the 128-byte swizzle
//    that the tensor cores read, and the scales.  Entries that select nothing
//    copy zeros; a tile without any entry costs no product.  (cp.async: a
//    gathering TMA copy of four rows takes 67 clocks to issue, 4300 a tile of
//    head_dim 128, where this takes 900.)
//  * an issuing warp: the output product of the oldest tile whose
//    probabilities are there, else the scores of a tile, at most two ahead:
//    accumulators of scores, buffers of probabilities and key stages take
//    turns in step, so one barrier each way serves all three.
//  * an epilogue warpgroup (thread = token): scores times the token's scale,
//    probability 2^(t - m), its sum per head in the thread, and P (times the
//    token's value scale) into shared memory as the next product's operand.
//    m goes by the largest P of the tile in which it was last set: a later
//    tile keeps it unless a P is 14 times as large, which takes one vote of the
//    group a tile instead of a maximum per head across its 128 threads.  A tile
//    that does not keep it takes the exact maxima, rescales the sums and the
//    accumulator and is done over.
// Many units: persistent CTAs, each pipeline with units of its own.  Few: a
// cluster of 1, 2, 4 or 8 CTAs per unit, whose pipelines share its tiles; their
// results meet in f32 through distributed shared memory.  Which one, by the
// tiles of the busiest SM, is decided on the host (api.cpp).
//
// What bounds it: with many query heads per key head, the softmax's latency (a
// tile of 32 heads takes a warpgroup about 2500 clocks, 1150 of them arithmetic, the
// rest waits, the vote and fences between roles; half of the issue slots are
// filled, the tensor cores are busy 14% of the time).  4096 prompt rows of 32
// heads and 2048 entries: 328 us, 419 TFLOP/s; a verify step of 96 such rows
// 22 us; 128 heads on one key head 21 us (500 to 600 GB/s through the gather).
// 8 heads a key head over pages of one token: the scattered rows, 1.3 GB through
// L2 in 244 us (182 us if the pages lie in order, 137 us with pages of 64
// tokens).  One decode row: latency, 9.2 us, of which two dependent loads before
// the first copy take 1.4 and the meeting of the cluster 2.
// Every wait is bounded (common.cuh).  After a wait has run out the group
// votes, so that its four warps leave together and no barrier is left open.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "operators.h"

namespace cg = cooperative_groups;

namespace fp8idx {

static __device__ unsigned int g_attn_watchdog;

namespace {

constexpr uint32_t kFull = 0xffffffffu;
// What is multiplied with a value's code is P = 2^(t - m) * kTopCode * vs / cref
// (t the score in log2 units, vs the value's scale).  P's codes reach from 448
// (the largest e4m3 value) down to steps of 2^-13 (the smallest one of the
// second part: 2^-9 / 16), so m goes by the products, not by the scores alone:
// it is the largest t + log2(vs / cref) of the tile in which it was last set,
// which then has the code 32 and the others steps of 2^-18 of it.  It is set
// anew when a P exceeds 448; with normally distributed scores a unit of 2048
// entries does that once, at its first tile.
// cref is the first tile's largest value scale over 2^16; one more than 2^80
// times cref becomes the new one.  Sums are of 2^(t - m), so log2(vs / cref) is
// taken as no less than -96: entries with values that small (or zero) and
// nearly all of the weight then have a 2^(t - m) of up to 2^96, and a thread's
// 16 of them a sum up to 2^104.
constexpr float kTopCode = 32.f, kMaxCode = 448.f;
constexpr float kOverFirst = 0x1p-16f, kMaxOver = 0x1p80f, kLogOver = 80.f, kMinOver = 0x1p-96f, kLogUnder = 96.f;
constexpr float kMaxSum = 0x1p104f, kHugeTerm = 0x1p126f;
constexpr float kMinVScale = 0x1p-120f;
constexpr float kMinM = -3e38f;       // m stays finite, so that a score of -inf gives probability 0

// One warp-collective bounded wait, in few instructions: this kernel has many
// roles, and their loops together have to stay in the instruction cache.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t site) {
  bool ok = ptx::mbar_test_wait(bar, parity);
  if (!ok) {
    const uint64_t since = ptx::globaltimer_ns();
#pragma unroll 1
    while (!(ok = ptx::mbar_try_wait(bar, parity))) {
      if (*abort_flag) break;
      if (ptx::globaltimer_ns() - since > kWaitTimeoutNs) {
        *abort_flag = 1u;
        atomicOr(&g_attn_watchdog, site);
        break;
      }
    }
  }
  return __all_sync(kFull, ok);
}

// Two at once: one round of tests in the usual case that both are complete.
__device__ __forceinline__ bool attn_wait2(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1,
                                           volatile uint32_t* abort_flag, uint32_t site0, uint32_t site1) {
  const bool a = ptx::mbar_test_wait(bar0, parity0), b = ptx::mbar_test_wait(bar1, parity1);
  if (__all_sync(kFull, a && b)) return true;
  return attn_wait(bar0, parity0, abort_flag, site0) && attn_wait(bar1, parity1, abort_flag, site1);
}

__device__ __forceinline__ bool attn_wait3(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, uint32_t bar2,
                                           uint32_t parity2, volatile uint32_t* abort_flag, uint32_t site0, uint32_t site1,
                                           uint32_t site2) {
  const bool a = ptx::mbar_test_wait(bar0, parity0), b = ptx::mbar_test_wait(bar1, parity1);
  const bool c = ptx::mbar_test_wait(bar2, parity2);
  if (__all_sync(kFull, a && b && c)) return true;
  return attn_wait(bar0, parity0, abort_flag, site0) && attn_wait(bar1, parity1, abort_flag, site1) &&
         attn_wait(bar2, parity2, abort_flag, site2);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where a unit's results go: elements from `out` and `lse` on, heads it has.
struct UnitPlace {
  int64_t out;
  int32_t lse, heads;
};
__device__ __forceinline__ UnitPlace place_of(const SparseAttnParams& p, int row, int head, int heads) {
  const int req = row / p.next_n;
  return {req * p.out_req_stride + (row - req * p.next_n) * p.out_row_stride + head * p.out_head_stride,
          row * p.heads + head, heads};
}

// Softmax state of a CTA in shared memory; NG epilogue groups.
template <int GP, int NG, int QB>
struct AttnState {
  UnitPlace qplace[QB];        // [query buffer]
  UnitPlace place[NG];         // [group]
  float nm[NG][GP];            // -m of each group (log2 units), 0 before a unit's first tile
  float ninf[GP];              // -inf: the row of -m that an entry without a token reads
  float part[NG][4][GP];       // [group][warp]: a tile's maxima over m; a unit's sums
  float resc[NG][GP];          // a new maximum: 2^-(half of what m grows by, which may be 200)
  float fac[NG][GP];           // a unit's end: factor of the accumulator
  float xl[NG][GP];            // cluster: log2 of the group's sum per head, its maximum included
  float wvs[NG][4];            // a tile's largest value scales
  float qf[QB];                // [query buffer]: 2^-e of the query's scaling
  uint32_t spread[QB];         // whether its heads have factors
  int8_t qhead[QB][GP], head[NG][4][GP];  // log2 of the heads' factors: [query buffer], [group][warp]
  uint32_t top[GP];            // cluster: largest element per head
  uint2 qpart[2][2];           // [queries take turns][query warp]: its heads' largest and lowest `top`
};

// A load that is issued where it stands: the compiler would otherwise sink a
// load whose value is needed in the loop's next turn past the copies.
__device__ __forceinline__ int32_t load_now(const int32_t* a) {
  int32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}

// Registers move from the copying and issuing warps to the epilogue's.
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Column j of N (16 or 32) columns, one value per lane and column: the lanes'
// maximum (or sum), in lane j (and j + 16 for N = 16).  N - 1 (+ 1) shuffles.
template <int N, bool MAX>
__device__ __forceinline__ float reduce_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int j = 0; j < d; ++j) {
      const float got = __shfl_xor_sync(kFull, up ? v[j] : v[j + d], d);
      const float own = up ? v[j + d] : v[j];
      v[j] = MAX ? fmaxf(own, got) : own + got;
    }
  }
  if constexpr (N == 16) {
    const float got = __shfl_xor_sync(kFull, v[0], 16);
    v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

constexpr uint32_t pow2_at_least(uint32_t n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

__device__ __forceinline__ void unit_of(const SparseAttnParams& p, int u, int* row, int* kvh, int* h0, int gp) {
  const int c = u / p.head_chunks;
  *h0 = (u - c * p.head_chunks) * gp;
  *row = c / p.kv_heads;
  *kvh = c - *row * p.kv_heads;
}

// Splits two values into e4m3 pairs h and l with x = h + l / 16.
__device__ __forceinline__ void split_pair(__half2 x, uint32_t* h, uint32_t* l) {
  const __nv_fp8x2_storage_t hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3));
  const __half2 r = __hmul2(__hsub2(x, back), __floats2half2_rn(16.f, 16.f));
  *h = hi;
  *l = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
}

// The query's split: every element of a unit times the 2^e that puts the
// unit's largest finite one into [128, 256), as two e4m3 values.  If the
// largest element of one of its heads lies below 16 then, every head gets an e
// of its own, and its scores the factor 2^(unit's e - its e).  So a head's
// elements are exact from 2^-6 on, 2^-10 of its largest one, and off by at
// most 2^-18 of that below (half a step of 2^-13).  Factors go down to 2^-126:
// where heads are further apart than that, the unit's e is so much larger, and
// its scores in the accumulator (at most 2^24 before) so much larger with it.
// It takes 96 at most: heads more than 2^222 below the largest, whose elements
// are below 2^-94, then have scores off by less than 2^-78 times the scales.
struct QueryPiece {
  uint32_t top;  // the largest element's bits without its sign (bf16 values are then ordered as integers)
  bool odd;      // infinities or NaN among them (from 0x7F80; they do not count)
  __device__ __forceinline__ explicit QueryPiece(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m2 = 0, s2 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = w[k] & 0x7FFF7FFFu, special = __vcmpgeu2(m, 0x7F807F80u);
      s2 |= special;
      m2 = __vmaxu2(m2, m & ~special);
    }
    top = max(m2 >> 16, m2 & 0xFFFFu);
    odd = s2 != 0u;
  }
};
__device__ __forceinline__ int query_exponent(uint32_t top) {
  const int e = 134 - static_cast<int>(top >> 7);
  return top == 0u ? 0 : min(max(e, -120), 120);
}
// The exponent of a head with largest element `top` (0: none) in a unit whose
// heads' are between `low` (of those that have one, else 0xFFFF) and `high`;
// unit_e: the unit's.
__device__ __forceinline__ int head_exponent(uint32_t top, uint32_t low, uint32_t high, bool* apart, int* unit_e) {
  const int e = query_exponent(high), gap = low != 0xFFFFu ? query_exponent(low) - e : 0;
  *apart = gap > 3;
  *unit_e = e + min(max(gap - 126, 0), 96);
  return *apart && top != 0u ? query_exponent(top) : *unit_e;
}
__device__ __forceinline__ uint32_t low_of(uint32_t top) { return top == 0u ? 0xFFFFu : top; }

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Eight elements of head g (16-byte piece `piece` of its row) into the two
// parts' rows: 128 bytes each, 128-byte swizzle.
template <int GP>
__device__ __forceinline__ void store_query(uint8_t* dst, int g, int piece, const uint4& v, float mul, bool odd) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, h[4], l[4];
  if (odd) {  // an infinity becomes NaN: as a code it would be the largest value
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] |= __vcmpeq2(w[k] & 0x7FFF7FFFu, 0x7F807F80u) & 0x7FFF7FFFu;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    split_pair(__floats2half2_rn(__uint_as_float(w[k] << 16) * mul, __uint_as_float(w[k] & 0xFFFF0000u) * mul), &h[k],
               &l[k]);
  const int chunk = piece >> 1, half = (piece & 1) * 8, r1 = g, r2 = GP + g;
  *reinterpret_cast<uint2*>(dst + r1 * 128 + ((chunk ^ (r1 & 7)) << 4) + half) =
      make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  *reinterpret_cast<uint2*>(dst + r2 * 128 + ((chunk ^ (r2 & 7)) << 4) + half) =
      make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

}  // namespace

template <int D, int GP, bool CLUSTER>
__global__ void __launch_bounds__(kAttnThreads, 1) sparse_attn_kernel(const __grid_constant__ SparseAttnParams p) {
  constexpr int NG = kAttnGroups;
  constexpr int kProdWarp0 = 4 * NG, kProdWarps = 4 * NG;
  constexpr int kMmaWarp0 = kProdWarp0 + kProdWarps, kQWarp = kMmaWarp0 + NG, kQWarps = 2;
  static_assert(32 * (kQWarp + kQWarps) == kAttnThreads, "roles");
  constexpr int N2 = 2 * GP;                       // columns of S^T and O^T
  constexpr int SBG = 2;                           // accumulators of S^T per group
  constexpr int QB = kAttnQueryBuffers, PB = kAttnProbBuffers;
  constexpr int KS = attn_k_stages(D), S = attn_v_stages(D);  // D = 64: keys and values share the rows of S
  constexpr int KSG = KS > 0 ? KS / NG : 1, SG = S / NG;         // a group's share
  static_assert(KS % NG == 0 && S % NG == 0 && SG >= SBG, "stages");
  static_assert(SBG == 2 && PB == 2 && (KS == 0 || KSG == SBG), "rings that go in step");
  constexpr uint32_t kTmemCols = pow2_at_least(NG * (SBG + 1) * N2);
  constexpr uint32_t kTmemO = NG * SBG * N2;       // O^T of group g at kTmemO + g * N2
  using State = AttnState<GP, NG, QB>;
  static_assert(sizeof(State) <= 4u * attn_state_floats(GP), "state");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_1024(smem_raw);
  constexpr AttnSmem L = attn_smem_layout(D, GP);
  static_assert(L.total <= kMaxSmem, "shared memory");
  State& stt = *reinterpret_cast<State*>(smem + L.flt);
  const uint32_t k0 = ptx::smem_u32(smem + L.k), v0 = ptx::smem_u32(smem + L.v);
  const uint32_t q0 = ptx::smem_u32(smem + L.q);
  const uint32_t full0 = ptx::smem_u32(smem + L.bars), empty0 = full0 + 8u * S;
  const uint32_t qf0 = empty0 + 8u * S, qe0 = qf0 + 8u * QB;                  // query buffers
  const uint32_t sf0 = qe0 + 8u * QB;                                         // [group][buffer] scores ready
  const uint32_t pf0 = sf0 + 8u * NG * SBG, pe0 = pf0 + 8u * NG * PB;         // [group][buffer] probabilities ready, used
  const uint32_t ub = pe0 + 8u * NG * PB, drain0 = ub + 8u;                   // cluster: both groups done; [MMA warp]
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L.misc);
  volatile uint32_t* abort_flag = misc + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    misc[1] = 0u;
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full0 + 8u * s, 33u * 4u);        // each producer lane's copies, each warp's mask
      ptx::mbar_init(empty0 + 8u * s, 1u);               // the output MMA
    }
    for (int i = 0; i < QB; ++i) {
      ptx::mbar_init(qf0 + 8u * i, CLUSTER ? 4u * NG : kQWarps);
      ptx::mbar_init(qe0 + 8u * i, 1u + 4u);             // the last score MMA, the unit's epilogue warps
    }
    for (int i = 0; i < NG * SBG; ++i) ptx::mbar_init(sf0 + 8u * i, 1u);
    for (int i = 0; i < NG * PB; ++i) {
      ptx::mbar_init(pf0 + 8u * i, 4u);
      ptx::mbar_init(pe0 + 8u * i, 1u);
    }
    ptx::mbar_init(ub, 4u * NG);
    for (int i = 0; i < NG; ++i) ptx::mbar_init(drain0 + 8u * i, 1u);
    ptx::fence_barrier_init();
  }
  for (int g = threadIdx.x; g < GP; g += kAttnThreads) stt.ninf[g] = -INFINITY, stt.top[g] = 0u;
  for (int g = threadIdx.x; g < NG * GP; g += kAttnThreads) stt.nm[g / GP][g % GP] = 0.f;
  if (warp == kMmaWarp0) {
    ptx::tmem_alloc(ptx::smem_u32(misc), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  // This CTA's work.  Each epilogue group has a producer set, an issuing warp
  // and rings of stages of its own: NG pipelines side by side that share
  // nothing but the query warps.  In a persistent CTA group g takes the units
  // g, g + NG, ... of the CTA's list; in a cluster's CTA, which has one unit,
  // every NG-th of its tiles.
  const int C = CLUSTER ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
  const int crank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int per = (p.tiles + C - 1) / C;
  const int t0 = min(crank * per, p.tiles), t1 = min(t0 + per, p.tiles);
  const int u0 = CLUSTER ? static_cast<int>(blockIdx.x) / C : static_cast<int>(blockIdx.x);
  const int ustep = static_cast<int>(gridDim.x);
  const int n_units = CLUSTER ? 1 : (p.units - u0 + ustep - 1) / ustep;
  const auto own_units = [&](int g) { return CLUSTER ? 1 : (n_units - g + NG - 1) / NG; };
  const auto unit_tiles = [&](int g) { return CLUSTER ? (t1 - t0 - g + NG - 1) / NG : t1 - t0; };

  if (warp >= 4 * NG) {
    reg_dec<kAttnOtherRegs>();
    if (warp < kMmaWarp0) {
      // =========================== producers ===========================
      // The four warps of a group's set copy its tiles, 32 entries each (a lane
      // resolves one).
      const int g = (warp - kProdWarp0) / 4;
      constexpr int kRowLanes = 2 * D / 16;                    // lanes that copy a token's 16-byte pieces
      constexpr int kRowsPerCopy = 32 / kRowLanes;
      const int tok0 = (warp - kProdWarp0) % 4 * 32;           // this warp's tokens of a tile
      const int shift = p.block_shift, in_page = p.block_size - 1;
      // Lane l copies piece l % kRowLanes of every kRowsPerCopy-th token into
      // its place in the 128-byte swizzle, which depends on the token mod 8.
      const int piece = lane % kRowLanes, sub = lane / kRowLanes;
      uint32_t place[8 / kRowsPerCopy];
#pragma unroll
      for (int i = 0; i < 8 / kRowsPerCopy; ++i)
        place[i] = (tok0 + sub) * 128 + (((piece & 7) ^ ((i * kRowsPerCopy + sub) & 7)) << 4);
      const uint8_t* const my_piece = p.kv + piece * 16;
      const uint32_t my_scale = ptx::smem_u32(smem + L.scale) + (tok0 + lane) * 8u;
      uint32_t* const my_mask = reinterpret_cast<uint32_t*>(smem + L.mask) + (tok0 >> 5);
      const int per_unit = unit_tiles(g), total = own_units(g) * per_unit;
      if (total > 0) {
        // Entries are loaded two tiles ahead of their copies, table entries one.
        // Offsets into the cache are 32-bit numbers of p.unit bytes.
        Ring st{0u, 0u, static_cast<uint32_t>(SG)}, kst{0u, 0u, static_cast<uint32_t>(KSG)};
        int32_t idx1 = -1, blk = -1, off = 0, req1 = 0, req2 = 0;
        uint32_t head = 0, head1 = 0, head2 = 0;
        // the look-ahead: the next tile's place, tiles left in its unit, the next unit
        const int32_t* at = nullptr;
        int room = 0, left = 0, unit = g;
        int req = 0;  // prefill: the request that the last column was found in
        int32_t req_lo = 0, req_hi = -1;
#pragma unroll 1
        for (int it = -2; it < total; ++it) {
          int32_t blk1 = -1, idx2 = -1, tok = idx1;
          {  // the next tile's table entries
            bool ok = tok >= 0;
            if (p.cu_seq_lens != nullptr) {
              if (ok && (tok < req_lo || tok >= req_hi)) {
                int a = 0, b = p.n_req;
#pragma unroll 1
                while (b - a > 1) {
                  const int mid = (a + b) >> 1;
                  if (__ldg(p.cu_seq_lens + mid) <= tok) a = mid; else b = mid;
                }
                req = a;
                req_lo = __ldg(p.cu_seq_lens + a);
                req_hi = __ldg(p.cu_seq_lens + a + 1);
              }
              ok = ok && tok >= req_lo && tok < req_hi;
              tok = static_cast<int32_t>(static_cast<uint32_t>(tok) - static_cast<uint32_t>(req_lo));
            } else {
              req = req1;
            }
            // (unsigned: lengths that are no prefix sums must not lead out of the table)
            const uint32_t j = static_cast<uint32_t>(tok >> shift);
            if (ok && j < static_cast<uint32_t>(p.max_blocks))
              blk1 = load_now(p.block_tables + static_cast<int64_t>(req) * p.bt_stride + j);
          }
          if (it + 2 < total) {  // the entries of the tile after that
            if (left == 0) {     // a new unit: taken apart once
              int row, kvh, h0;
              unit_of(p, u0 + (CLUSTER ? 0 : unit) * ustep, &row, &kvh, &h0, GP);
              const int first = (t0 + (CLUSTER ? g : 0)) * kAttnTile + tok0 + lane;
              at = p.indices + row * p.idx_stride + first;
              room = p.k - first;
              req2 = row / p.next_n;
              head2 = kvh * p.head_units;
              left = per_unit;
              unit += NG;
            }
            if (room > 0) idx2 = load_now(at);
            at += (CLUSTER ? NG : 1) * kAttnTile;
            room -= (CLUSTER ? NG : 1) * kAttnTile;
            --left;
          }
          if (it >= 0) {
            const bool ok = blk >= 0 && blk < p.num_blocks;
            const uint32_t m = __ballot_sync(kFull, ok);
            const uint32_t page = head + static_cast<uint32_t>(blk) * p.block_units;
            const uint32_t from = page + static_cast<uint32_t>(off) * p.tok_units;
            const uint32_t stage = g * SG + st.idx, k_stage = g * KSG + kst.idx;
            // (a key stage is free once the scores of the tile in it are: their buffers take turns like the stages)
            if (KS > 0 ? !attn_wait2(empty0 + 8u * stage, st.phase ^ 1u, sf0 + 8u * k_stage, kst.phase ^ 1u, abort_flag,
                                     kSiteStageEmpty, kSiteAccFull)
                       : !attn_wait(empty0 + 8u * stage, st.phase ^ 1u, abort_flag, kSiteStageEmpty))
              break;
            const uint32_t full = full0 + 8u * stage;
            const uint32_t at_stage = KS > 0 && piece < 8 ? k0 + k_stage * kAttnHalfBytes : v0 + stage * kAttnHalfBytes;
            if (ok)
              ptx::cp_async_8(my_scale + stage * (kAttnTile * 8u),
                              p.kv + static_cast<uint64_t>(page) * p.unit + (p.scale_off + 8 * off));
            if (lane == 0) my_mask[4 * stage] = m;
            if (m == kFull) {
              uint32_t f[32 / kRowsPerCopy];  // (all shuffles first: none waits for a copy to be issued)
#pragma unroll
              for (int j = 0; j < 32 / kRowsPerCopy; ++j) f[j] = __shfl_sync(kFull, from, j * kRowsPerCopy + sub);
#pragma unroll
              for (int j = 0; j < 32; j += kRowsPerCopy)
                ptx::cp_async_16(at_stage + place[(j & 7) / kRowsPerCopy] + j * 128u,
                                 my_piece + static_cast<uint64_t>(f[j / kRowsPerCopy]) * p.unit);
            } else {  // entries without a token copy zeros
#pragma unroll 1
              for (int j = 0; j < 32; j += kRowsPerCopy) {
                const uint32_t f = __shfl_sync(kFull, from, j + sub);
                const bool valid = m >> (j + sub) & 1u;
                const uint32_t dst = at_stage + (tok0 + j + sub) * 128u + (((piece ^ (j + sub)) & 7) << 4);
                ptx::cp_async_16_zfill(dst, valid ? my_piece + static_cast<uint64_t>(f) * p.unit : p.kv, valid ? 16u : 0u);
              }
            }
            ptx::cp_async_mbar_arrive(full);
            if (lane == 0) ptx::mbar_arrive(full);
            st.next();
            kst.next();
          }
          blk = blk1, off = tok & in_page, head = head1;
          idx1 = idx2, req1 = req2, head1 = head2;
        }
        ptx::cp_async_wait_all();  // (an abandoned call must not leave copies behind)
      }
    } else if (warp >= kQWarp) {
      // =========================== queries =============================
      // Two warps, half of the unit's heads each: kHeads rows a round, kPer
      // lanes a row, and after a reduction of all rounds together lane l has
      // the largest element of head head_of.
      constexpr int kPer = D / 8, kHeads = 32 / kPer, kRounds = GP / kQWarps / kHeads;
      const int w = warp - kQWarp, head_of = lane % kPer % kRounds * kHeads + lane / kPer;
#pragma unroll 1
      for (int i = 0; !CLUSTER && i < n_units; ++i) {  // (a cluster's epilogue warps do it)
        const int buf = i % QB;
        int row, kvh, h0;
        unit_of(p, u0 + i * ustep, &row, &kvh, &h0, GP);
        const int nh = min(GP, p.group - h0), first = w * (GP / kQWarps);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row / p.next_n * p.q_req_stride +
                                 row % p.next_n * p.q_row_stride + (kvh * p.group + h0) * p.q_head_stride;
        uint4 v[kRounds];
        uint32_t t[kRounds];
        bool odd = false;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const int h = first + r * kHeads + lane / kPer;
          v[r] = make_uint4(0u, 0u, 0u, 0u);
          if (h < nh) v[r] = __ldg(reinterpret_cast<const uint4*>(q + h * p.q_head_stride + lane % kPer * 8));
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const QueryPiece piece(v[r]);
          t[r] = piece.top;
          odd |= piece.odd;
        }
#pragma unroll
        for (int d = kRounds / 2; d > 0; d >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int j = 0; j < d; ++j) {
            const uint32_t got = __shfl_xor_sync(kFull, up ? t[j] : t[j + d], d);
            t[j] = max(up ? t[j + d] : t[j], got);
          }
        }
#pragma unroll
        for (int d = kRounds; d < kPer; d *= 2) t[0] = max(t[0], __shfl_xor_sync(kFull, t[0], d));
        const uint32_t high = __reduce_max_sync(kFull, t[0]), low = __reduce_min_sync(kFull, low_of(t[0]));
        odd = __any_sync(kFull, odd);
        if (lane == 0) stt.qpart[i & 1][w] = make_uint2(high | (odd ? 0x10000u : 0u), low);
        const bool ok = attn_wait(qe0 + 8u * buf, ((i / QB) & 1) ^ 1, abort_flag, kSiteQEmpty);
        if (ptx::bar_or(2 + NG, 32 * kQWarps, !ok)) break;
        const uint2 x = stt.qpart[i & 1][0], y = stt.qpart[i & 1][1];
        odd = ((x.x | y.x) & 0x10000u) != 0u;
        const uint32_t top = max(x.x & 0xFFFFu, y.x & 0xFFFFu);
        bool apart;
        int unit_e;
        const int e = head_exponent(t[0], min(x.y, y.y), top, &apart, &unit_e);
        stt.qhead[buf][first + head_of] = static_cast<int8_t>(max(unit_e - e, -126));
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const float mul = power_of_two(__shfl_sync(kFull, e, lane / kPer * kPer + r));  // (lane of the row's head)
          store_query<GP>(smem + L.q + buf * N2 * 128, first + r * kHeads + lane / kPer, lane % kPer, v[r], mul, odd);
        }
        if (w == 0 && lane == 0) {
          stt.qf[buf] = power_of_two(-unit_e);
          stt.spread[buf] = apart;
          stt.qplace[buf] = place_of(p, row, kvh * p.group + h0, nh);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(qf0 + 8u * buf);
      }
    } else {
      // ============================= MMA ===============================
      // A warp per group issues its products: the output of the oldest tile
      // whose probabilities are there, else the scores of a tile (two ahead
      // at most: their accumulators take turns).  The whole warp walks the
      // tiles (its values stay uniform), one lane issues.
      const int g = warp - kMmaWarp0;
      constexpr uint32_t kIdescS = ptx::idesc_e4m3_f32(kAttnTile, N2);
      constexpr uint32_t kIdescO = ptx::idesc_e4m3_f32(128, N2) | ptx::kIdescMnMajorA | ptx::kIdescMnMajorB;
      const uint64_t sa0 = ptx::smem_desc_sw128(KS > 0 ? k0 : v0), sb0 = ptx::smem_desc_sw128(q0);
      const uint64_t oa0 = ptx::smem_desc_mn(v0, 128);
      const uint64_t ob = ptx::smem_desc_mn(ptx::smem_u32(smem + L.p) + g * PB * kAttnTile * N2, N2);
      Ring ss{0u, 0u, static_cast<uint32_t>(SG)}, so = ss;
      const int per_unit = unit_tiles(g), own = own_units(g) * per_unit;
      int is = 0, io = 0, left_s = per_unit, left_o = per_unit;  // tiles scored, put out; left in the unit
      int unit_s = CLUSTER ? 0 : g;
      uint32_t live = 0;              // [is & 1]: whether a scored tile has entries
      bool first = true;              // the unit's first output starts the accumulator anew
      uint64_t since = 0;
      uint32_t spins = 0;
#pragma unroll 1
      while (io < own) {
        if (io < is) {
          const uint32_t buf = io & 1, bar = 8u * (g * PB + buf);
          if (__all_sync(kFull, ptx::mbar_test_wait(pf0 + bar, (io >> 1) & 1))) {
            // (the group makes its next unit's first probabilities after it has read the last unit's outputs)
            ptx::tc_fence_after();
            const bool any = live >> buf & 1u;
            const uint32_t stage = g * SG + so.idx;
            const uint64_t a = oa0 + static_cast<uint64_t>(stage * (kAttnHalfBytes >> 4));
            const uint64_t b = ob + static_cast<uint64_t>(buf * (kAttnTile * N2 >> 4));
            if (ptx::elect_one()) {
              if (any) {
#pragma unroll
                for (int kk = 0; kk < kAttnTile / 32; ++kk)
                  ptx::mma_f8f6f4(tmem + kTmemO + g * N2, a + kk * (32ull * 128 >> 4), b + kk * (32ull * N2 >> 4), kIdescO,
                                  (first && kk == 0) ? 0u : 1u);
              }
              ptx::mma_commit(pe0 + bar);
              ptx::mma_commit(empty0 + 8u * stage);
            }
            __syncwarp();
            first = first && !any;
            ++io;
            so.next();
            if (--left_o == 0) {
              left_o = per_unit;
              first = true;
            }
            spins = 0;
            continue;
          }
        }
        if (is < own && is < io + SBG && __all_sync(kFull, ptx::mbar_test_wait(full0 + 8u * (g * SG + ss.idx), ss.phase))) {
          const int buf = unit_s % QB;
          if (left_s == per_unit && !attn_wait(qf0 + 8u * buf, (unit_s / QB) & 1, abort_flag, kSiteQFull)) break;
          const uint32_t stage = g * SG + ss.idx, slot = g * SBG + (is & 1);
          const uint4 m = *reinterpret_cast<const uint4*>(smem + L.mask + 16 * stage);
          const bool any = (m.x | m.y | m.z | m.w) != 0u;
          live = (live & ~(1u << (is & 1))) | static_cast<uint32_t>(any) << (is & 1);
          ptx::fence_proxy_async_smem();  // the tile was written by cp.async
          ptx::tc_fence_after();
          const uint64_t a = sa0 + static_cast<uint64_t>((KS > 0 ? slot : stage) * (kAttnHalfBytes >> 4));
          const uint64_t b = sb0 + static_cast<uint64_t>(buf * (N2 * 128u >> 4));
          if (ptx::elect_one()) {
            if (any) {
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                ptx::mma_f8f6f4(tmem + slot * N2, a + 2ull * kk, b + 2ull * kk, kIdescS, kk > 0 ? 1u : 0u);
            }
            ptx::mma_commit(sf0 + 8u * slot);
            if (left_s == 1) ptx::mma_commit(qe0 + 8u * buf);  // the unit's last tile
          }
          __syncwarp();
          ++is;
          ss.next();
          if (--left_s == 0) {
            left_s = per_unit;
            unit_s += NG;
          }
          spins = 0;
          continue;
        }
        if ((++spins & 63u) == 0u) {
          bool give_up = *abort_flag != 0u;
          const uint64_t now = ptx::globaltimer_ns();
          if (spins == 64u) since = now;
          if (now - since > kWaitTimeoutNs) {
            give_up = true;
            *abort_flag = 1u;
            if (lane == 0) atomicOr(&g_attn_watchdog, static_cast<uint32_t>(kSiteAccEmpty));
          }
          if (__any_sync(kFull, give_up)) break;
        }
      }
      __syncwarp();
      if (*abort_flag && lane == 0) {
        const uint32_t bar = drain0 + 8u * g;
        ptx::mma_commit(bar);
        wait_drain(bar, 0, &g_attn_watchdog);
      }
      __syncwarp();
    }
  } else {
    // ============================ epilogue =============================
    reg_inc<kAttnEpilogueRegs>();
    const int g = warp >> 2, quad = warp & 3;
    const int tg = threadIdx.x & 127;                 // thread in the group = token = channel
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_tm = tmem + kTmemO + g * N2 + lane_off;
    uint8_t* const p_rows = smem + L.p + g * PB * kAttnTile * N2 + tg * N2;
    // 16-byte chunks of a row of probabilities, swizzled over its N2 bytes
    const uint32_t p_swz = N2 == 64 ? (tg >> 1) & 3 : (tg >> 2) & 1;
    const int bar_id = 1 + g;
    Ring st{0u, 0u, static_cast<uint32_t>(SG)};
    uint32_t n = 0;                                   // this group's tiles so far
    bool stop = false;
    // the output MMA of the last tile before this one (they complete in order)
    const auto wait_outputs = [&] {
      attn_wait(pe0 + 8u * (g * PB + ((n - 1u) & 1u)), ((n - 1u) >> 1) & 1u, abort_flag, kSiteAccEmpty);
      ptx::tc_fence_after();
    };
    if (CLUSTER && t0 < t1) {
      // The unit's query: nothing else is to be done yet, and 256 threads have
      // it ready by the time the first tile is.
      int row, kvh, h0;
      unit_of(p, u0, &row, &kvh, &h0, GP);
      const int nh = min(GP, p.group - h0);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row / p.next_n * p.q_req_stride +
                               row % p.next_n * p.q_row_stride + (kvh * p.group + h0) * p.q_head_stride;
      constexpr int kPer = D / 8, kPieces = (GP * kPer + 255) / 256;
      uint4 v[kPieces];
      bool odd = false;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = static_cast<int>(threadIdx.x) + 256 * i;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c < nh * kPer) v[i] = __ldg(reinterpret_cast<const uint4*>(q + c / kPer * p.q_head_stride + c % kPer * 8));
        const QueryPiece piece(v[i]);
        if (c < GP * kPer) atomicMax(&stt.top[c / kPer], piece.top);
        odd |= piece.odd;
      }
      odd = ptx::bar_or(1 + NG, 4 * NG * 32, odd);
      const uint32_t top = lane < GP ? stt.top[lane % GP] : 0u, high = __reduce_max_sync(kFull, top);
      bool apart;
      int unit_e;
      const int e = head_exponent(top, __reduce_min_sync(kFull, low_of(top)), high, &apart, &unit_e);
      if (threadIdx.x < GP) stt.qhead[0][threadIdx.x] = static_cast<int8_t>(max(unit_e - e, -126));
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = static_cast<int>(threadIdx.x) + 256 * i, head = min(c / kPer, GP - 1);
        const float mul = power_of_two(__shfl_sync(kFull, e, head));
        if (c < GP * kPer) store_query<GP>(smem + L.q, head, c % kPer, v[i], mul, odd);
      }
      if (threadIdx.x == 0) {
        stt.qf[0] = power_of_two(-unit_e);
        stt.spread[0] = apart;
        stt.qplace[0] = place_of(p, row, kvh * p.group + h0, nh);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(qf0);
    }
    if (CLUSTER && t0 >= t1 && threadIdx.x == 0) {  // (a CTA without tiles finishes heads as well)
      int row, kvh, h0;
      unit_of(p, u0, &row, &kvh, &h0, GP);
      stt.qplace[0] = place_of(p, row, kvh * p.group + h0, min(GP, p.group - h0));
    }
#pragma unroll 1
    for (int r = 0; r < own_units(g) && !stop; ++r) {
      const int unit = CLUSTER ? 0 : r * NG + g;
      float qscale = 0.f;
      bool ok = true, spread = false;
      if (t0 < t1) {
        ok = attn_wait(qf0 + 8u * (unit % QB), (unit / QB) & 1, abort_flag, kSiteQFull);
        qscale = stt.qf[unit % QB] * p.scale_log2;
        spread = stt.spread[unit % QB] != 0u;
        if (lane < GP) stt.head[g][quad][lane] = stt.qhead[unit % QB][lane];
        if (!CLUSTER && tg == 0) stt.place[g] = stt.qplace[unit % QB];  // (read between the unit's last two barriers)
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(qe0 + 8u * (unit % QB));
      }
      uint32_t has_o = 0u;  // whether the group's accumulator holds anything of this unit
      float cref = 0.f, wref = 0.f;  // the value scales' reference, kTopCode over it
      float2 l2[GP / 2];
#pragma unroll
      for (int j = 0; j < GP / 2; ++j) l2[j] = make_float2(0.f, 0.f);

#pragma unroll 1
      for (int left = unit_tiles(g); left > 0; --left) {
        const uint32_t stage = g * SG + st.idx, stage_phase = st.phase;
        st.next();
        asm volatile("" : "+r"(has_o));  // (one copy of the loop: the first tile is not peeled off)
        // (accumulators of scores and buffers of probabilities take turns alike)
        const uint32_t buf = n & 1u, parity = (n >> 1) & 1u;
        const uint32_t slot = g * SBG + buf, pbar = 8u * (g * PB + buf);
        uint8_t* const p_row = p_rows + buf * kAttnTile * N2;
        ok = attn_wait3(full0 + 8u * stage, stage_phase, sf0 + 8u * slot, parity, pe0 + pbar, parity ^ 1u, abort_flag,
                        kSiteStageFull, kSiteAccFull, kSiteAccEmpty) && ok;
        ptx::tc_fence_after();
        const uint32_t s_tm = tmem + slot * N2 + lane_off;
        if (spread) {  // heads far apart: their factors go into the accumulator, out of the way of the usual case
#pragma unroll 1
          for (int b = 0; b < N2; b += 16) {
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(s_tm + b, v);
            ptx::tmem_wait_ld_n(v);
            const int8_t* f = &stt.head[g][quad][b % GP];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * power_of_two(f[j]));
            ptx::tmem_st_32x32b_x16(s_tm + b, v);
          }
          ptx::tmem_wait_st();
        }
        // The scores of the first 16 heads (of no meaning in a tile without
        // entries); 32 heads need the registers (early: 342 us, late: 333 us).
        uint32_t hi[16], lo[16];
        if constexpr (GP == 16) {
          ptx::tmem_ld_32x32b_x16(s_tm, hi);
          ptx::tmem_ld_32x32b_x16(s_tm + GP, lo);
        }
        const uint4 mk = *reinterpret_cast<const uint4*>(smem + L.mask + 16 * stage);
        const bool any = (mk.x | mk.y | mk.z | mk.w) != 0u;
        const uint32_t mw = quad == 0 ? mk.x : quad == 1 ? mk.y : quad == 2 ? mk.z : mk.w;
        const bool valid = mw >> lane & 1u;
        const float2 sc = reinterpret_cast<const float2*>(smem + L.scale)[stage * kAttnTile + tg];
        const float c = valid ? sc.x * qscale : 0.f;
        const float vs = valid ? sc.y : 0.f;
        const float4* nm4 = reinterpret_cast<const float4*>(valid ? stt.nm[g] : stt.ninf);
        // scores of heads b .. b+15 over the present m, in log2 units
        const auto scores = [&](int b, const uint32_t (&hi)[16], const uint32_t (&lo)[16], float (&t)[16]) {
          const float2 c2 = make_float2(c, c), k16 = make_float2(0.0625f, 0.0625f);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 nm = nm4[(b + j) / 4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float2 raw = __ffma2_rn(make_float2(__uint_as_float(lo[j + k]), __uint_as_float(lo[j + k + 1])), k16,
                                            make_float2(__uint_as_float(hi[j + k]), __uint_as_float(hi[j + k + 1])));
              const float2 t2 = __ffma2_rn(raw, c2, k == 0 ? make_float2(nm.x, nm.y) : make_float2(nm.z, nm.w));
              t[j + k] = t2.x;
              t[j + k + 1] = t2.y;
            }
          }
        };
        if constexpr (GP == 16) {
          ptx::tmem_wait_ld_n(hi);
          ptx::tmem_wait_ld_n(lo);
        }
        // The probabilities are computed and stored against the m in hand; if
        // one of them shows that m is too small (or m is not set yet), the
        // group takes the maxima and does them over.
#pragma unroll 1
        for (bool fresh = false;; fresh = true) {
          bool again = any && !has_o && !fresh;
          if (any && (has_o || fresh)) {
            const float w = vs * wref;
            const float2 w2 = make_float2(w, w);
            __half2 top = __floats2half2_rn(0.f, 0.f);
            float t[16];
            if constexpr (GP > 16) {
              ptx::tmem_ld_32x32b_x16(s_tm, hi);
              ptx::tmem_ld_32x32b_x16(s_tm + GP, lo);
              ptx::tmem_wait_ld_n(hi);
              ptx::tmem_wait_ld_n(lo);
            }
            scores(0, hi, lo, t);
#pragma unroll
            for (int b = 0; b < GP; b += 16) {
              uint32_t ph[4], pl[4];
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                uint32_t hc[2], lc[2];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const float2 e = make_float2(ex2(t[j + k]), ex2(t[j + k + 1]));
                  float2& l = l2[(b + j + k) / 2];
                  l = __fadd2_rn(l, e);
                  const float2 pf = __fmul2_rn(e, w2);
                  const __half2 p2 = __floats2half2_rn(pf.x, pf.y);  // (11 bits; above 65504 infinite, which is caught)
                  top = __hmax2(top, __habs2(p2));
                  split_pair(p2, &hc[k / 2], &lc[k / 2]);
                }
                ph[j / 4] = hc[0] | hc[1] << 16;
                pl[j / 4] = lc[0] | lc[1] << 16;
              }
              *reinterpret_cast<uint4*>(p_row + (((b / 16) ^ p_swz) << 4)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
              *reinterpret_cast<uint4*>(p_row + ((((GP + b) / 16) ^ p_swz) << 4)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
              if (b + 16 < GP) {
                uint32_t hi1[16], lo1[16];
                ptx::tmem_ld_32x32b_x16(s_tm + b + 16, hi1);
                ptx::tmem_ld_32x32b_x16(s_tm + GP + b + 16, lo1);
                ptx::tmem_wait_ld_n(hi1);
                ptx::tmem_wait_ld_n(lo1);
                scores(b + 16, hi1, lo1, t);
              }
            }
            ptx::fence_proxy_async_smem();  // (before the vote, which hides some of its wait)
            again = fabsf(w) > kTopCode * kMaxOver || !__hble2(top, __floats2half2_rn(kMaxCode, kMaxCode));
            if (valid && !(fabsf(w) >= kTopCode * kMinOver)) {  // a scale so small (or NaN) that P does not bound the sums
              float sum = 0.f;
#pragma unroll
              for (int j = 0; j < GP / 2; ++j) sum = fmaxf(sum, fmaxf(l2[j].x, l2[j].y));
              again |= sum > kMaxSum;
            }
            again = again && !fresh;
          }
          // (every warp votes in every pass: an abandoned call may have left them with different masks)
          if (!ptx::bar_or(bar_id, 128, again || !ok)) break;
          // ---- new maxima
          const float vmax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(fabsf(vs))));
          if (lane == 0) stt.wvs[g][quad] = vmax;
          if (ptx::bar_or(bar_id, 128, !ok)) {  // an abandoned call: all four warps leave
            stop = true;
            break;
          }
          const float last_cref = cref;
          {
            const float m = fmaxf(fmaxf(stt.wvs[g][0], stt.wvs[g][1]), fmaxf(stt.wvs[g][2], stt.wvs[g][3]));
            if (!has_o || m > kMaxOver * cref) cref = fmaxf(m * kOverFirst, kMinVScale);
            wref = kTopCode / cref;
          }
          {
            const float lv = fminf(fmaxf(__log2f(fabsf(vs)) - __log2f(cref), -kLogUnder), kLogOver);
            float v[GP];
#pragma unroll
            for (int b = 0; b < GP; b += 16) {
              uint32_t h[16], l[16];
              ptx::tmem_ld_32x32b_x16(s_tm + b, h);
              ptx::tmem_ld_32x32b_x16(s_tm + GP + b, l);
              ptx::tmem_wait_ld_n(h);
              ptx::tmem_wait_ld_n(l);
              scores(b, h, l, *reinterpret_cast<float(*)[16]>(&v[b]));
            }
            if (has_o) {  // take the tile's sums back (what a huge one leaves is nothing beside it)
#pragma unroll
              for (int j = 0; j < GP / 2; ++j) {
                const float ex = ex2(v[2 * j]), ey = ex2(v[2 * j + 1]);
                l2[j] = make_float2(ex < kHugeTerm ? l2[j].x - ex : 0.f, ey < kHugeTerm ? l2[j].y - ey : 0.f);
              }
            }
#pragma unroll
            for (int j = 0; j < GP; ++j) v[j] += lv;
            const float t = reduce_columns<GP, true>(v, lane);
            if (lane < GP) stt.part[g][quad][lane] = t;
          }
          ptx::bar_sync(bar_id, 128);
          if (tg < GP) {
            const float d = fmaxf(fmaxf(fmaxf(stt.part[g][0][tg], stt.part[g][1][tg]),
                                        fmaxf(stt.part[g][2][tg], stt.part[g][3][tg])),
                                  has_o ? 0.f : kMinM);
            stt.resc[g][tg] = ex2(-0.5f * d);
            stt.nm[g][tg] -= d;
          }
          ptx::bar_sync(bar_id, 128);
          if (has_o) {
            wait_outputs();
#pragma unroll
            for (int j = 0; j < GP / 2; ++j) {
              const float2 f = *reinterpret_cast<const float2*>(&stt.resc[g][2 * j]);
              l2[j] = make_float2(l2[j].x * f.x * f.x, l2[j].y * f.y * f.y);
            }
            const float cf = last_cref / cref;
#pragma unroll 1
            for (int b = 0; b < N2; b += 16) {
              uint32_t v[16];
              ptx::tmem_ld_32x32b_x16(o_tm + b, v);
              ptx::tmem_wait_ld_n(v);
              const float* f = &stt.resc[g][b % GP];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * (f[j] * f[j] * cf));
              ptx::tmem_st_32x32b_x16(o_tm + b, v);
            }
            ptx::tmem_wait_st();
          }
        }
        if (stop) break;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(pf0 + pbar);  // (of a tile without entries: that it has been looked at)
        has_o |= any;
        ++n;
      }
      if (stop) break;

      // ---- the unit's end: the sums over the group's tokens, and the output
      {
        float v[GP];
#pragma unroll
        for (int j = 0; j < GP; j += 2) v[j] = l2[j / 2].x, v[j + 1] = l2[j / 2].y;
        const float sum = reduce_columns<GP, false>(v, lane);
        if (lane < GP) stt.part[g][quad][lane] = sum;
      }
      ptx::bar_sync(bar_id, 128);
      const UnitPlace pl = stt.place[g];  // (a cluster's outputs go out further down)
      const int nh = pl.heads;
      if (tg < GP) {
        const float sum = (stt.part[g][0][tg] + stt.part[g][1][tg]) + (stt.part[g][2][tg] + stt.part[g][3][tg]);
        const float m = has_o ? -stt.nm[g][tg] : kMinM;
        stt.nm[g][tg] = 0.f;
        stt.fac[g][tg] = sum == 0.f ? 0.f : cref / (sum * kTopCode);
        if constexpr (CLUSTER)
          stt.xl[g][tg] = sum == 0.f ? -INFINITY : m + log2f(sum);
        else if (p.lse != nullptr && tg < nh)
          p.lse[pl.lse + tg] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      }
      if (has_o) wait_outputs();
      if constexpr (CLUSTER) {  // the outputs go where the tiles were: both groups are done with them
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ub);
        attn_wait(ub, 0, abort_flag, kSiteAccFull);
      }
      ptx::bar_sync(bar_id, 128);
      const int ch = D == 128 ? tg : tg - 64;  // D = 64: the value half of the shared rows
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + pl.out + ch;
      float* xo = reinterpret_cast<float*>(smem + L.k) + g * GP * 128 + tg;  // cluster: [group][GP][128]
#pragma unroll 1
      for (int b = 0; b < GP; b += 16) {
        float v[16];
        if (has_o) {
          uint32_t hi[16], lo[16];
          ptx::tmem_ld_32x32b_x16(o_tm + b, hi);
          ptx::tmem_ld_32x32b_x16(o_tm + GP + b, lo);
          ptx::tmem_wait_ld_n(hi);
          ptx::tmem_wait_ld_n(lo);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = fmaf(__uint_as_float(lo[j]), 0.0625f, __uint_as_float(hi[j])) * stt.fac[g][b + j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0.f;
        }
        if constexpr (CLUSTER) {
#pragma unroll
          for (int j = 0; j < 16; ++j) xo[(b + j) * 128] = v[j];
        } else if (ch >= 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (b + j < nh) *out = __float2bfloat16(v[j]);
            out += p.out_head_stride;
          }
        }
      }
      ptx::tc_fence_before();  // (ordered before the barrier of the next unit's first probabilities)
    }
  }

  if constexpr (CLUSTER) {
    // ---- the groups of every CTA meet: CTA r finishes heads [r*GP/C, (r+1)*GP/C)
    cg::cluster_group cl = cg::this_cluster();
    const auto meet = [&] {
      __syncwarp();
      if (C > 1) cl.sync(); else __syncthreads();
    };
    meet();
    const int R = C * NG, heads = GP / C, first = crank * heads;  // partial results, heads of this CTA
    if (warp < 4 * NG) {  // (the others have few registers left)
      const UnitPlace pl = stt.qplace[0];
      const int nh = pl.heads;
      // thread (head, r), r fastest: the factor of partial result r
      if (threadIdx.x < GP * NG) {
        const int r = static_cast<int>(threadIdx.x) % R, h = first + static_cast<int>(threadIdx.x) / R;
        const float l_r = *cl.map_shared_rank(&stt.xl[r % NG][h], r / NG);
        const uint32_t lanes = GP * NG < 32 ? (1u << (GP * NG % 32)) - 1u : kFull;
        float m = fmaxf(l_r, kMinM);
        for (int d = R / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, d));
        const float f = ex2(l_r - m);  // (NaN for a partial result that is)
        float sum = f;
        for (int d = R / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(lanes, sum, d);
        (&stt.fac[0][0])[threadIdx.x] = sum == 0.f ? 0.f : __fdividef(f, sum);
        if (p.lse != nullptr && r == 0 && h < nh)
          p.lse[pl.lse + h] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      }
      ptx::bar_sync(1 + NG, 4 * NG * 32);
      // a warp per head, four channels a lane
      const int ch = 4 * lane - (D == 128 ? 0 : 64);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + pl.out + ch;
      const uint32_t xo = ptx::smem_u32(smem + L.k) + 16u * lane;
#pragma unroll 1
      for (int i = warp; i < heads; i += 4 * NG) {
        const int h = first + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < R; ++r) {
          const float f = (&stt.fac[0][0])[i * R + r];
          const float4 x = ptx::ld_cluster_f4(ptx::map_rank(xo + (r % NG * GP + h) * 512u, r / NG));
          v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
        }
        if (h < nh && ch >= 0) {
          __nv_bfloat16* o = out + h * p.out_head_stride;
          o[0] = __float2bfloat16(v.x), o[1] = __float2bfloat16(v.y);
          o[2] = __float2bfloat16(v.z), o[3] = __float2bfloat16(v.w);
        }
      }
    }
    meet();  // no CTA leaves while another reads its shared memory
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

namespace {
using AttnKernel = void (*)(SparseAttnParams);
template <int D, bool CLUSTER>
AttnKernel attn_instance(int gp) {
  return gp == 16 ? sparse_attn_kernel<D, 16, CLUSTER> : sparse_attn_kernel<D, 32, CLUSTER>;
}
}  // namespace

cudaError_t launch_sparse_attn(const SparseAttnParams& p, int head_dim, int grid, int ctas,
                               int smem_bytes, cudaStream_t stream) {
  const int gp = attn_pad(p.group);
  const AttnKernel kern = head_dim == 128 ? (ctas > 0 ? attn_instance<128, true>(gp) : attn_instance<128, false>(gp))
                                          : (ctas > 0 ? attn_instance<64, true>(gp) : attn_instance<64, false>(gp));
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem_bytes);
  if (e != cudaSuccess) return e;
  if (ctas == 0) {
    kern<<<grid, kAttnThreads, smem_bytes, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kAttnThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t read_attn_watchdog(unsigned int* value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_attn_watchdog, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_attn_watchdog, &zero, sizeof(unsigned int));
}

}  // namespace fp8idx
