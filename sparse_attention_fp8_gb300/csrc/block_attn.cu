// Dense attention over a paged e4m3 cache whose blocks share one scale
// (fp8_paged_block_attn) for sm_103a.
//
//   s[r, j] = softmax_scale * <q[r], K[j]>,  out[r] = sum_j softmax(s)[r, j] V[j]
//
// A unit is one key head and up to 256 query rows (positions x its query heads)
// of one request; its positions are taken in tiles of 128.  Both products run
// on the tensor cores with a query row per accumulator lane:
//   S [128 rows x 128 tokens] = [Qh | Ql] * [K | K]^T     (e4m3: the cache's bytes)
//   O [128 rows x D]         += P * V                     (f16: P from tensor memory)
// A query is split once a unit into two e4m3 values, x 2^e = h + l, which hold
// bf16's 8 bits; both products go into one accumulator.  P has 11 bits as f16,
// and V's codes become f16, exactly, in shared memory: a conversion for each
// value byte and 256 rows, where splitting P as well would cost four for each
// score.
//
// A CTA (16 warps) walks its units with
//  * two softmax warpgroups, one accumulator of scores and one of outputs each;
//    a thread has one row, so its maximum and sum need no other thread.  More
//    than 128 rows: each group has half of the rows and both see every tile.
//    Up to 128: both have the same rows and take the tiles in turn; up to 64 or
//    32, the rows stand in a tile's lanes twice or four times, and each copy
//    takes that share of the tile's tokens: its other probabilities are zeros.
//    The copies' results meet through shared memory at the unit's end.
//  * a converting warpgroup: V's codes to f16, NaN codes to zeros and a mask of
//    their tokens, so that they reach the rows that see them and no others.
//  * a warp that loads pages by TMA and the blocks' scales, two tiles ahead of
//    them their table entries; one that issues the products; one that walks the
//    units.
// The units' steps (a tile for both groups, or two tiles) are dealt out evenly:
// every CTA takes an equal range of them, from lengths on the device.  A unit
// that several CTAs share leaves its pieces in the workspace, and a second
// kernel joins them.
// The reference of a row goes by the products 2^t * vscale (t the score in log2
// units), so that P, which is multiplied with codes, keeps its bits: the largest
// one of its first tile, raised when one could exceed 2^15 times that.  Sums are
// of unrounded f32 exponentials.
// Every wait is bounded (common.cuh); a role whose wait has run out leaves, and
// then so do the others.
//
// What bounds it, measured with replayed graphs (the join included):
//  * 32 requests of one row, 64 / 8 heads, 32768 positions: 341 us, 5.4 TB/s of
//    cache, 81% of a copy's rate (one cache over and over; 374 to 385 over several).  A tile's 32 KB take 1420 clocks of an SM's
//    share of that rate, its products 1024 of the tensor pipe, for 8 rows as for
//    128, and its softmax and conversion have to stay below as well.
//  * 16 requests of 6 rows, 32 heads on one key head, 131072 positions: 198 us,
//    892 TFLOP/s; 4 requests of 2048 prompt rows, 32 / 8 heads, 8192 positions:
//    577 us, 1135 TFLOP/s, 58% of a bf16 product's rate.  The 1024 clocks of a
//    tile and 128 rows are half scores (e4m3, but twice: both parts of a query)
//    and half outputs (f16); the tensor pipe is busy 47% and the issue slots 44%
//    of the time (2 x 1024 rows): the chain of a tile - scores, softmax,
//    probabilities, outputs - is what takes the time, with two in flight.  The
//    code of the roles' inner loops has to stay within the instruction cache:
//    loops are rolled and what is rare is out of line (unrolled softmax 924 us
//    where the rolled one took 861).
//  * the prompts with heads of 64: 500 us, 655 TFLOP/s.
//  * one row of 1024 positions: 15.4 us, 2.5 of it the join: launch, plan, table
//    entry, scales, tile, one step and the meeting are one chain.
// Queries in tensor memory with scores in halves of a tile (887 us where this
// took 802), all scores of a tile held in registers (1203 against 820) and both
// chunks loaded ahead (717 against 640) were slower.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "operators.h"

namespace fp8idx {

static __device__ unsigned int g_block_attn_watchdog;

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kTile = 128;
constexpr int kConvWarp0 = 8, kLoadWarp = 12, kMmaWarp = 13, kPlanWarp = 14;
// Registers a thread: 256 * 184 + 128 * 80 + 128 * 64 = 512 * 128.
constexpr int kSoftmaxRegs = 184, kConvRegs = 80, kOtherRegs = 64;
constexpr float kMinM = -3e38f;   // m stays finite, so that a score of -inf gives probability 0
// A group of scale 0 (or NaN) has weights and no values: log2 of its scale counts as this far below the
// largest one of the piece so far, where its exponentials neither vanish beside the others' (below 2^-126)
// nor raise the reference over them.
constexpr float kNoScaleLog = -64.f;
// Bounds of the logarithms, so that their inverses and sums stay finite.
constexpr float kMinScaleLog = -100.f, kMaxScaleLog = 126.f;
// (Scale slots outnumber the tiles in flight: a tile's masks of NaN stay behind it
// until its group has looked, two of its tiles later.)
constexpr int kUnitSlots = 8, kScaleSlots = 8;
constexpr int kUnitCost = 4;      // a unit's start and end, in steps (3 to 8 are within 2% of one another)

// A CTA's share of a unit.
struct Piece {
  int32_t row0;        // first row; -1: no more pieces
  int32_t positions;   // rows / heads per key head
  int32_t head;        // key head
  int32_t req;
  int32_t pos0;        // position of the first row
  int32_t len;         // positions that exist
  int32_t ta, tb;      // tiles
  int32_t shared;      // both groups see every tile
  int32_t slot;        // -1: the whole unit, else the workspace piece
};

// Scales of a tile: per 16 tokens the keys' (times the softmax's), log2 of the
// values' over `ref` and its inverse; bits of groups of 16 tokens without
// values (0-7), with values that are NaN (8-15), in the cache (16-23), with a
// negative key scale (24-31).
struct TileScales {
  float key[8], vlog[8], vinv[8];
  float ref;
  uint32_t flags, pad[2];
  uint4 nan;           // (by the converting warps) tokens with a NaN among their values
};
static_assert(sizeof(TileScales) == 128, "a scale slot");

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 3 : 6;       // tiles in flight
  static constexpr uint32_t kHalf = kTile * 128u;         // a tile's keys or values (D 64: both)
  static constexpr uint32_t q = 0;                        // [group]; group 1's is also where copies meet
  static constexpr uint32_t qBytes = 2u * kHalf;          // of a group (the meeting takes 32 KB)
  static constexpr uint32_t k = q + 2 * qBytes;
  static constexpr uint32_t v = k + (D == 128 ? kStages * kHalf : 0);
  static constexpr uint32_t v16 = v + kStages * kHalf;    // two tiles of f16 values
  static constexpr uint32_t kV16 = kTile * D * 2u;
  static constexpr uint32_t scales = v16 + 2 * kV16;
  static constexpr uint32_t units = scales + kScaleSlots * sizeof(TileScales);
  static constexpr uint32_t bars = units + kUnitSlots * 64u;
  // barriers
  static constexpr uint32_t kFullB = bars, kEmptyB = kFullB + 8 * kStages;
  static constexpr uint32_t vFullB = kEmptyB + 8 * kStages, vEmptyB = vFullB + 8 * kStages;
  static constexpr uint32_t scaleFullB = vEmptyB + 8 * kStages, v16FullB = scaleFullB + 8 * kScaleSlots;  // by tile % kScaleSlots
  static constexpr uint32_t v16EmptyB = v16FullB + 8 * kScaleSlots;
  static constexpr uint32_t qFullB = v16EmptyB + 16, sFullB = qFullB + 16, pFullB = sFullB + 16, oFullB = pFullB + 16;
  static constexpr uint32_t unitFullB = oFullB + 16, unitEmptyB = unitFullB + 8 * kUnitSlots;
  static constexpr uint32_t meetB = unitEmptyB + 8 * kUnitSlots, drainB = meetB + 8;
  static constexpr uint32_t misc = drainB + 8;            // tensor memory's address, abort flag
  static constexpr uint32_t total = misc + 16 + 1024;     // and the alignment
};
static_assert(Smem<128>::kStages < kScaleSlots && Smem<64>::kStages < kScaleSlots, "scale slots");
static_assert(Smem<128>::total <= kMaxSmem && Smem<64>::total <= kMaxSmem, "shared memory");
static_assert(sizeof(Piece) <= 64, "a unit slot");
// The plan's prefix sums lie where the f16 values and the scales will.
static_assert((kMaxBatch + 1) * 8 <= 2 * Smem<64>::kV16 + kScaleSlots * sizeof(TileScales), "prefix sums");

// One warp-collective bounded wait.
__device__ __forceinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t site) {
  bool ok;
  const uint64_t since = ptx::globaltimer_ns();
#pragma unroll 1
  while (!(ok = ptx::mbar_try_wait(bar, parity))) {
    if (*abort_flag) break;
    if (ptx::globaltimer_ns() - since > kWaitTimeoutNs) {
      *abort_flag = 1u;
      atomicOr(&g_block_attn_watchdog, site);
      break;
    }
  }
  return __all_sync(kFull, ok);
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t site) {
  if (__all_sync(kFull, ptx::mbar_test_wait(bar, parity))) return true;
  return wait_longer(bar, parity, abort_flag, site);
}

// The same for a thread alone.
__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t site) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  return wait_bounded(bar, parity, abort_flag, &g_block_attn_watchdog, site);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------- the plan
// A request's rows and positions.  (Clamped: lengths that are no prefix sums
// must not lead out of the tensors.)
struct Request {
  int32_t row0, rows;  // rows
  int64_t pos0;        // of the first row
  int32_t len;         // positions that exist
  __device__ __forceinline__ Request(const BlockAttnParams& p, int b) {
    const int32_t a = __ldg(p.cu_new + b), e = __ldg(p.cu_new + b + 1), ctx = __ldg(p.context_lens + b);
    row0 = min(max(a, 0), p.rows);
    rows = max(min(e, p.rows) - row0, 0);
    pos0 = static_cast<int64_t>(ctx) - e + row0;
    len = static_cast<int32_t>(min(static_cast<int64_t>(max(ctx, 0)), static_cast<int64_t>(p.max_blocks) << p.block_shift));
  }
};
// Unit u of a request: its positions (rows / heads), tiles and steps.
struct Unit {
  int32_t at, positions, pos0, ta, tb, steps;
  bool shared;
  __device__ __forceinline__ Unit(const BlockAttnParams& p, const Request& r, int u) {
    const int half = p.half_positions;
    at = u * 2 * half;
    positions = min(2 * half, r.rows - at);
    shared = positions > half;
    const int64_t first = r.pos0 + at, last = first + positions - 1;
    const int32_t hi = static_cast<int32_t>(min(max(last + 1, static_cast<int64_t>(0)), static_cast<int64_t>(r.len)));
    const int32_t lo = p.window > 0 ? static_cast<int32_t>(min(max(first - p.window + 1, static_cast<int64_t>(0)),
                                                               static_cast<int64_t>(r.len)))
                                    : 0;
    ta = lo / kTile;
    tb = max((hi + kTile - 1) / kTile, ta + 1);  // (rows that see nothing take one tile, all masked)
    steps = shared ? tb - ta : (tb - ta + 1) / 2;
    pos0 = static_cast<int32_t>(max(first, static_cast<int64_t>(-(1 << 30))));  // (none reaches context_lens[b])
  }
};
__device__ __forceinline__ int unit_count(const BlockAttnParams& p, const Request& r) {
  return (r.rows + 2 * p.half_positions - 1) / (2 * p.half_positions);
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// --------------------------------------------------------------- the softmax
// Which of the 32 columns from `col` on (of the tile at `tile0`) a row at
// position pos sees.
__device__ __forceinline__ uint32_t seen32(int pos, int window, int len, int tile0, int col, uint32_t in_cache) {
  const int past = pos + 1 - tile0 - col, hi = min(past, len - tile0 - col);
  const int lo = window > 0 ? max(past, 0) - window : 0;  // (no difference leaves 32 bits)
  uint32_t m = hi <= 0 ? 0u : hi >= 32 ? kFull : (1u << hi) - 1u;
  if (lo > 0) m &= lo >= 32 ? 0u : kFull << lo;
  if (!(in_cache >> (col / 16) & 1u)) m &= 0xFFFF0000u;
  if (!(in_cache >> (col / 16 + 1) & 1u)) m &= 0x0000FFFFu;
  return m;
}

// Whether a row sees a NaN in the chunks chunk0 .. end of the last n tiles (each
// `step` after the other) before tile j, which starts at tile0.
__device__ __noinline__ bool sees_nan(const TileScales* scales, uint32_t j, int tile0, int step, int n, int chunk0, int end,
                                      int pos, int window, int len) {
  uint32_t seen = 0;
#pragma unroll 1
  for (int back = 1; back <= n; ++back) {
    const uint32_t* const words = reinterpret_cast<const uint32_t*>(&scales[(j - back * step) % kScaleSlots].nan);
#pragma unroll 1
    for (int c = chunk0; c < end; ++c) seen |= words[c] & seen32(pos, window, len, tile0 - back * step * kTile, c * 32, 0xFFu);
  }
  return seen != 0u;
}

struct RowState {
  float m = kMinM, l = 0.f;
  bool bad = false;  // sees a value that is NaN
};

// What turns 32 scores (two groups of 16) into log2 probabilities x c + o, and
// the groups' inverse value scales.  Masked scores are log2 probabilities.
struct ChunkScale {
  float2 c, o, vinv;
  __device__ __forceinline__ ChunkScale(const TileScales& sc, int k, bool masked, float row_scale) {
    const float2 key = reinterpret_cast<const float2*>(sc.key)[k];
    c = masked ? make_float2(1.f, 1.f) : make_float2(key.x * row_scale, key.y * row_scale);
    o = masked ? make_float2(0.f, 0.f) : reinterpret_cast<const float2*>(sc.vlog)[k];
    vinv = reinterpret_cast<const float2*>(sc.vinv)[k];
  }
};
__device__ __forceinline__ float chunk_max(const uint32_t (&r)[32], const ChunkScale& cs) {
  float top = -INFINITY;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t* v = &r[16 * g];
    float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]);
#pragma unroll
    for (int j = 2; j < 16; j += 4) {
      a = fmaxf(fmaxf(a, __uint_as_float(v[j])), __uint_as_float(v[j + 1]));
      if (j + 2 < 16) b = fmaxf(fmaxf(b, __uint_as_float(v[j + 2])), __uint_as_float(v[j + 3]));
    }
    top = fmaxf(top, fmaf(fmaxf(a, b), g ? cs.c.y : cs.c.x, g ? cs.o.y : cs.o.x));
  }
  return top;
}
// Probabilities of 32 scores over 2^m, as f16 pairs; their sum is added to `most`.
// Returns the sum over the value scales.
__device__ __forceinline__ float chunk_exp(const uint32_t (&r)[32], const ChunkScale& cs, float m, uint32_t (&h)[16],
                                           float& most) {
  float l = 0.f;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float c = g ? cs.c.y : cs.c.x, o = (g ? cs.o.y : cs.o.x) - m;
    const float2 cc = make_float2(c, c), oo = make_float2(o, o);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[16 * g + j]), __uint_as_float(r[16 * g + j + 1])), cc, oo);
      const float2 e = make_float2(ex2(x.x), ex2(x.y));
      sum = __fadd2_rn(sum, e);
      const __half2 hv = __floats2half2_rn(e.x, e.y);
      h[g * 8 + j / 2] = *reinterpret_cast<const uint32_t*>(&hv);
    }
    const float s = sum.x + sum.y;
    most += s;
    l = fmaf(s, g ? cs.vinv.y : cs.vinv.x, l);
  }
  return l;
}

// Of a tile that not every row sees in full, or where a key scale is negative (the
// largest score is not the largest probability's then): log2 probabilities, -inf
// where the row sees nothing, in the scores' place.
__device__ __noinline__ void mask_tile(uint32_t s_tm, const TileScales* sc, int chunk0, int end, int pos, int window, int len,
                                       int tile0, float row_scale) {
#pragma unroll 1
  for (int k = chunk0; k < end; ++k) {
    uint32_t r[32];
    ptx::tmem_ld_32x32b_x32(s_tm + k * 32, r);
    const uint32_t see = seen32(pos, window, len, tile0, k * 32, sc->flags >> 16);
    ptx::tmem_wait_ld_regs(r);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float x = fmaf(__uint_as_float(r[j]), sc->key[2 * k + j / 16] * row_scale, sc->vlog[2 * k + j / 16]);
      r[j] = __float_as_uint(see >> j & 1u ? x : -INFINITY);
    }
    ptx::tmem_st_32x32b_x32(s_tm + k * 32, r);
  }
  ptx::tmem_wait_st();
}

// A row's outputs times f.
template <int D>
__device__ __noinline__ void scale_outputs(uint32_t o_tm, float f) {
#pragma unroll 1
  for (int k = 0; k < D; k += 32) {
    uint32_t r[32];
    ptx::tmem_ld_32x32b_x32(o_tm + k, r);
    ptx::tmem_wait_ld_regs(r);
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
    ptx::tmem_st_32x32b_x32(o_tm + k, r);
  }
}

// Raises a row's reference to the largest log2 probability of the chunks k to
// end, rounded up (so that factors are powers of two), and scales what goes by
// the old one: the outputs (if there are any) and the tile's probabilities
// before chunk k.  Returns the new reference.
template <int D>
__device__ __noinline__ float raise_reference(uint32_t s_tm, uint32_t o_tm, const TileScales* sc, int chunk0, int k, int end,
                                              bool masked, float row_scale, bool outputs, float m) {
  float top = -INFINITY;
#pragma unroll 1
  for (int i = k; i < end; ++i) {
    uint32_t r[32];
    ptx::tmem_ld_32x32b_x32(s_tm + i * 32, r);
    ptx::tmem_wait_ld_regs(r);
    top = fmaxf(top, chunk_max(r, ChunkScale(*sc, i, masked, row_scale)));
  }
  const float now = fmaxf(m, ceilf(top)), f = ex2(m - now);
#pragma unroll 1
  for (int i = chunk0; i < k; ++i) {
    uint32_t h[16];
    ptx::tmem_ld_32x32b_x16(s_tm + i * 16, h);
    ptx::tmem_wait_ld_n(h);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const __half2 w = __floats2half2_rn(v.x * f, v.y * f);
      h[j] = *reinterpret_cast<const uint32_t*>(&w);
    }
    ptx::tmem_st_32x32b_x16(s_tm + i * 16, h);
  }
  if (outputs) scale_outputs<D>(o_tm, f);
  ptx::tmem_wait_st();
  return now;
}

// A tile's scores to probabilities, `chunks` (1, 2 or 4) times 32 columns from
// chunk0 on; the rest of the probabilities are zeros.  Probabilities lie over
// the scores (16 columns for 32), written in order, so those of a chunk
// overwrite scores that have been read.  No maximum is looked for: the sum of a
// pair of chunks shows whether its probabilities stay within f16 (each below
// 2^15); where one does not, and at a row's first tile, the reference is raised
// and the pair done over.  (A pass for the maximum took a third of the
// instructions.)  The loop is rolled: unrolled it waits for its instructions,
// as the roles' loops together do not fit the instruction cache then.
template <int D>
__device__ __forceinline__ void softmax_tile(uint32_t s_tm, uint32_t o_tm, const TileScales& sc, int chunk0, int chunks,
                                             bool masked, int pos, int window, int len, int tile0, float row_scale, bool first,
                                             RowState& st) {
  const int end = chunk0 + chunks;
  if (masked) mask_tile(s_tm, &sc, chunk0, end, pos, window, len, tile0, row_scale);
  bool raised = false;
  const auto raise = [&](int k) {
    const float m = raise_reference<D>(s_tm, o_tm, &sc, chunk0, k, end, masked, row_scale, !first, st.m);
    st.l *= ex2(st.m - m);
    st.m = m;
    raised = true;
  };
  if (chunks > 1) {
#pragma unroll 1
    for (int k = chunk0; k < end;) {
      uint32_t r[32], h0[16], h1[16];
      float most = 0.f, l;
      ptx::tmem_ld_32x32b_x32(s_tm + k * 32, r);
      {
        const ChunkScale cs(sc, k, masked, row_scale);
        ptx::tmem_wait_ld_regs(r);
        l = chunk_exp(r, cs, st.m, h0, most);
      }
      ptx::tmem_ld_32x32b_x32(s_tm + (k + 1) * 32, r);
      {
        const ChunkScale cs(sc, k + 1, masked, row_scale);
        ptx::tmem_wait_ld_regs(r);
        l += chunk_exp(r, cs, st.m, h1, most);
      }
      if (__any_sync(kFull, !(most < 32768.f)) && !raised) {
        raise(k);
        continue;
      }
      st.l += l;
      ptx::tmem_st_32x32b_x16(s_tm + k * 16, h0);
      ptx::tmem_st_32x32b_x16(s_tm + (k + 1) * 16, h1);
      k += 2;
    }
  } else {
    uint32_t r[32], h[16];
    float l, most;
    while (true) {
      most = 0.f;
      ptx::tmem_ld_32x32b_x32(s_tm + chunk0 * 32, r);
      const ChunkScale cs(sc, chunk0, masked, row_scale);
      ptx::tmem_wait_ld_regs(r);
      l = chunk_exp(r, cs, st.m, h, most);
      if (!__any_sync(kFull, !(most < 32768.f)) || raised) break;
      raise(chunk0);
    }
    st.l += l;
    ptx::tmem_st_32x32b_x16(s_tm + chunk0 * 16, h);
  }
  if (chunks < 4) {
    const uint32_t zeros[16] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < chunk0 || k >= end) ptx::tmem_st_32x32b_x16(s_tm + k * 16, zeros);
  }
}

// ------------------------------------------------------------------ queries
// The 2^e that puts a row's largest finite element, with the bits `top`, into
// [128, 256).
__device__ __forceinline__ int query_exponent(uint32_t top) {
  const int e = 134 - static_cast<int>(top >> 7);
  return top == 0u ? 0 : min(max(e, -120), 120);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Two values as e4m3 pairs h and l with x = h + l.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t* h, uint32_t* l) {
  const __half2 x = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3));
  *h = hi;
  *l = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(x, back)), __NV_SATFINITE, __NV_E4M3);
}

// A group's query row r (zeros where q is null), of which its lanes have `copies`
// copies `apart` lanes apart: each thread writes every copies-th 16 elements of
// both parts, from its own copy's number on, for all of them (none if `write` is
// false).  Returns 2^-e.  D 128: h in rows of 128 bytes, l in a second tile; D 64:
// h and l in one row.  `sign` flips every element.
template <int D>
__device__ __forceinline__ float load_query(uint8_t* dst, int r, int copy, int copies, int apart, const __nv_bfloat16* q,
                                            bool write, uint32_t sign) {
  const uint4* const piece = reinterpret_cast<const uint4*>(q);
  uint32_t top2 = 0, odd = 0;
  if (q) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint4 v = __ldg(piece + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = w[k] & 0x7FFF7FFFu, special = __vcmpgeu2(m, 0x7F807F80u);  // infinities and NaN do not count
        odd |= special;
        top2 = __vmaxu2(top2, m & ~special);
      }
    }
  }
  const int e = query_exponent(max(top2 >> 16, top2 & 0xFFFFu));
  if (write) {
    const float mul = __uint_as_float(__float_as_uint(power_of_two(e)) | sign);
    uint4 next[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (q) next[0] = __ldg(piece + 2 * copy), next[1] = __ldg(piece + 2 * copy + 1);
#pragma unroll 1
    for (int c = copy; c < D / 16; c += copies) {
      const uint4 v[2] = {next[0], next[1]};
      if (q && c + copies < D / 16) next[0] = __ldg(piece + 2 * (c + copies)), next[1] = __ldg(piece + 2 * (c + copies) + 1);
      uint32_t h[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4& x = v[i / 4];
        uint32_t w = i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w;
        // an infinity becomes NaN: as a code it would be the largest value
        if (odd) w |= __vcmpeq2(w & 0x7FFF7FFFu, 0x7F807F80u) & 0x7FFF7FFFu;
        split_pair(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xFFFF0000u) * mul, &h[i], &l[i]);
      }
      const int cl = D == 64 ? c + 4 : c;
      uint8_t* row = dst + r * 128;  // (rows `apart` lanes apart agree in the swizzle's bits)
#pragma unroll 1
      for (int k = 0; k < copies; ++k, row += apart * 128) {
        *reinterpret_cast<uint4*>(row + ((c ^ (r & 7)) << 4)) =
            make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        *reinterpret_cast<uint4*>(row + (D == 64 ? 0 : kTile * 128) + ((cl ^ (r & 7)) << 4)) =
            make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
      }
    }
  }
  return power_of_two(-e);
}

// Four e4m3 codes as f16.
__device__ __forceinline__ void half_pairs(uint32_t codes, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(codes));
}

// Where a lane's codes of a tile lie: eight lanes convert 64 codes of two
// tokens whose rows differ in bits 0 and 2, so that neither their reads nor
// their writes share banks.  Combination i * 4 + quarter of a panel of 64
// channels and a pair of rows.
template <int D>
struct ConvPlace {
  static constexpr int kPanels = D / 64, kTimes = 4 * kPanels;
  int w, piece, other, quarter;  // w: the warp's 32 tokens of a tile
  __device__ __forceinline__ ConvPlace(int warp, int lane)
      : w(warp), piece(lane & 3), other(lane >> 2 & 1), quarter(lane >> 3) {}
  __device__ __forceinline__ int panel(int i) const { return (i * 4 + quarter) % kPanels; }
  __device__ __forceinline__ int row(int i) const {
    const int pair = (i * 4 + quarter) / kPanels;
    return 32 * w + 8 * (pair >> 2) + ((pair & 3) ^ (other * 5));
  }
  __device__ __forceinline__ uint4 load(const uint8_t* src, int i) const {
    const int r = row(i), c = (D == 64 ? 4 : panel(i) * 4) + piece;
    return *reinterpret_cast<const uint4*>(src + r * 128 + ((c ^ (r & 7)) << 4));
  }
  __device__ __forceinline__ void store(uint8_t* dst, int i, const uint4& codes) const {
    const int r = row(i);
    uint32_t h[8];
    half_pairs(codes.x, &h[0], &h[1]);
    half_pairs(codes.y, &h[2], &h[3]);
    half_pairs(codes.z, &h[4], &h[5]);
    half_pairs(codes.w, &h[6], &h[7]);
    uint8_t* const at = dst + panel(i) * (kTile * 128) + r * 128;
    *reinterpret_cast<uint4*>(at + (((2 * piece) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at + (((2 * piece + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
  }
};

// A tile once more, with zeros for codes that are NaN and for groups of tokens
// whose scale is zero or NaN (flags).  Returns the warp's tokens with a NaN.
template <int D>
__device__ __noinline__ uint32_t convert_odd(uint8_t* dst, const uint8_t* src, int warp, int lane, uint32_t flags) {
  const ConvPlace<D> at(warp, lane);
  uint32_t nan_rows = 0;
#pragma unroll 1
  for (int i = 0; i < ConvPlace<D>::kTimes; ++i) {
    const uint4 x = at.load(src, i);
    const int r = at.row(i);
    const uint32_t group = flags >> (r >> 4);
    const bool none = ((group | group >> 8) & 1u) != 0u;
    uint32_t any = group >> 8 & 1u;
    const auto clear = [&](uint32_t v) {
      const uint32_t n = __vcmpeq4(v & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      any |= n;
      return none ? 0u : v & ~n;
    };
    at.store(dst, i, make_uint4(clear(x.x), clear(x.y), clear(x.z), clear(x.w)));
    if (any != 0u) nan_rows |= 1u << (r & 31);
  }
  return __reduce_or_sync(kFull, nan_rows);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    block_attn_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ BlockAttnParams p) {
  using L = Smem<D>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = align_up_1024(smem_raw);
  const uint32_t base = ptx::smem_u32(smem);
  uint32_t* const misc = reinterpret_cast<uint32_t*>(smem + L::misc);
  volatile uint32_t* const abort_flag = misc + 1;
  volatile uint32_t* const odd_values = misc + 2;  // a tile had a NaN among its values
  TileScales* const tile_scales = reinterpret_cast<TileScales*>(smem + L::scales);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto bar = [&](uint32_t at, int i = 0) { return base + at + 8u * i; };

  if (threadIdx.x == 0) {
    misc[1] = misc[2] = 0u;
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(bar(L::kFullB, s), 1u);
      ptx::mbar_init(bar(L::kEmptyB, s), D == 128 ? 1u : 5u);  // the score MMA (and the converting warps)
      ptx::mbar_init(bar(L::vFullB, s), 1u);
      ptx::mbar_init(bar(L::vEmptyB, s), 4u);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(L::v16EmptyB, i), 1u);
      ptx::mbar_init(bar(L::qFullB, i), 4u);
      ptx::mbar_init(bar(L::sFullB, i), 1u);
      ptx::mbar_init(bar(L::pFullB, i), 4u);
      ptx::mbar_init(bar(L::oFullB, i), 1u);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      ptx::mbar_init(bar(L::scaleFullB, i), 1u);
      ptx::mbar_init(bar(L::v16FullB, i), 4u);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      ptx::mbar_init(bar(L::unitFullB, i), 1u);
      ptx::mbar_init(bar(L::unitEmptyB, i), 1u + 1u + 4u + 8u);
    }
    ptx::mbar_init(bar(L::meetB), 8u);
    ptx::mbar_init(bar(L::drainB), 1u);
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(misc), 512);
    ptx::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) ptx::prefetch_tmap(&tm_kv);

  // ---- This CTA's range of steps: a key head's steps of each request, summed up.
  int64_t* const warp_sum = reinterpret_cast<int64_t*>(smem + L::q);
  int64_t* const cum = reinterpret_cast<int64_t*>(smem + L::v16);  // [n_req + 1], per key head
  {
    const int per = (p.n_req + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b >= p.n_req) break;
      const Request r(p, b);
      const int n = unit_count(p, r);
      int64_t steps = 0;
      if (n <= 16) {
        for (int u = 0; u < n; ++u) steps += Unit(p, r, u).steps + kUnitCost;
      } else {
        steps = -1;  // many units: a warp's work
      }
      cum[b + 1] = steps;
    }
    __syncthreads();
    for (int b = warp; b < p.n_req; b += kThreads / 32) {
      if (cum[b + 1] >= 0) continue;
      const Request r(p, b);
      const int n = unit_count(p, r);
      int64_t steps = 0;
      for (int u = lane; u < n; u += 32) steps += Unit(p, r, u).steps + kUnitCost;
      steps = __shfl_sync(kFull, warp_scan(steps, lane), 31);
      __syncwarp();
      if (lane == 0) cum[b + 1] = steps;
    }
    __syncthreads();
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b < p.n_req) mine += cum[b + 1];
    }
    const int64_t scan = warp_scan(mine, lane);
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int64_t before = scan - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b >= p.n_req) break;
      before += cum[b + 1];
      cum[b + 1] = before;
    }
    if (threadIdx.x == 0) cum[0] = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  // The plan warp finds the start of the range before the sums are overwritten.
  int64_t at = 0, end = 0, per_cta = 1;
  int req = 0, head = 0, unit = 0;
  int32_t skip = 0;  // steps of the first unit that earlier CTAs have
  if (warp == kPlanWarp) {
    const int64_t all = cum[p.n_req] * p.kv_heads;
    per_cta = max((all + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(1));
    at = min(blockIdx.x * per_cta, all);
    end = min(at + per_cta, all);
    if (at < end) {
      int hi = p.n_req;
      while (hi - req > 1) {
        const int mid = (req + hi) >> 1;
        if (cum[mid] * p.kv_heads <= at) req = mid; else hi = mid;
      }
      const int64_t steps = cum[req + 1] - cum[req], in = at - cum[req] * p.kv_heads;
      head = static_cast<int>(in / steps);
      int64_t rest = in - head * steps;
      const Request r(p, req);
      const int n = unit_count(p, r);
      for (unit = 0; unit < n; unit += 32) {  // 32 units at a time
        const int u = unit + lane;
        const int64_t sum = warp_scan(u < n ? Unit(p, r, u).steps + kUnitCost : 0, lane);
        const uint32_t over = __ballot_sync(kFull, sum > rest);
        if (over) {
          const int l = __ffs(over) - 1;
          const int64_t prev = __shfl_sync(kFull, sum, max(l - 1, 0));
          rest -= l > 0 ? prev : 0;
          unit += l;
          break;
        }
        rest -= __shfl_sync(kFull, sum, 31);
      }
      skip = static_cast<int32_t>(min(rest, static_cast<int64_t>(0x7fffffff)));
    }
  }
  __syncthreads();

  const auto slot_of = [&](uint32_t n) { return reinterpret_cast<Piece*>(smem + L::units + 64u * (n % kUnitSlots)); };
  // Reads piece n, once it is there.
  const auto get_piece = [&](uint32_t n, Piece* out) {
    if (!wait(bar(L::unitFullB, n % kUnitSlots), (n / kUnitSlots) & 1u, abort_flag, kSiteQEmpty)) return false;
    *out = *slot_of(n);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(L::unitEmptyB, n % kUnitSlots));
    return out->row0 >= 0;
  };

  if (warp >= kLoadWarp) {
    reg_dec<kOtherRegs>();
    if (warp == kPlanWarp) {
      // ============================ the plan ============================
      // (Lengths are read again here.  If someone writes them meanwhile, they need not be the ones the sums
      // were made of: every request, unit, step and piece stays in range all the same.)
      BlockAttnMeta meta = {};
      if (at < end) {
        Request r(p, req);
        int n_units = unit_count(p, r);
        uint32_t n = 0;
        bool ok = true;
#pragma unroll 1
        while (ok) {
          Piece out;
          out.row0 = -1;
          bool empty = false;
          if (at < end) {
            const Unit u(p, r, unit);
            const int32_t all = u.steps + kUnitCost;
            skip = min(skip, all);
            const int32_t stop = static_cast<int32_t>(min(static_cast<int64_t>(all), skip + (end - at)));
            // (the unit's cost stands before its steps)
            const int32_t from = max(skip - kUnitCost, 0), to = max(stop - kUnitCost, 0);
            empty = from == to;
            out.row0 = r.row0 + u.at;
            out.positions = u.positions;
            out.head = head;
            out.req = req;
            out.pos0 = u.pos0;
            out.len = r.len;
            out.shared = u.shared;
            out.ta = u.ta + (u.shared ? from : 2 * from);
            out.tb = min(u.ta + (u.shared ? to : 2 * to), u.tb);
            out.slot = from > 0 ? 0 : to < u.steps ? 1 : -1;
            if (out.slot == 1 && !empty) {
              meta.row0 = out.row0;
              meta.positions = out.positions;
              meta.head = head;
              meta.last = static_cast<int32_t>(min((at - skip + all - 1) / per_cta, static_cast<int64_t>(gridDim.x - 1)));
              meta.shared = out.shared;
            }
            at += stop - skip;
            skip = 0;
          }
          if (!empty) {
            ok = wait(bar(L::unitEmptyB, n % kUnitSlots), ((n / kUnitSlots) & 1u) ^ 1u, abort_flag, kSiteAccEmpty);
            if (!ok) break;
            if (lane == 0) {
              *slot_of(n) = out;
              ptx::mbar_arrive(bar(L::unitFullB, n % kUnitSlots));
            }
            __syncwarp();
            ++n;
          }
          if (out.row0 < 0) break;
          if (at < end && ++unit >= n_units) {
            unit = 0;
            if (++head == p.kv_heads) {
              head = 0;
              do {
                if (++req == p.n_req) at = end;
                r = Request(p, min(req, p.n_req - 1));
                n_units = unit_count(p, r);
              } while (n_units == 0 && at < end);
            }
          }
        }
      } else {
        if (lane == 0) {
          slot_of(0)->row0 = -1;
          ptx::mbar_arrive(bar(L::unitFullB, 0));
        }
      }
      if (lane == 0) p.meta[blockIdx.x] = meta;
    } else if (warp == kLoadWarp) {
      // ============================ the loads ============================
      // Lane l < 8 has the 16 tokens l of a tile: its block's table entry two
      // tiles ahead, its scales one.  A block that no row of the unit sees (past
      // its positions or before its window) counts as one outside the cache: its
      // bytes and scales may be anything.
      struct Ahead {
        int32_t block = -1, head = 0, first = 0, live = 0;
      };
      const int shift = p.block_shift;
      Piece piece;
      uint32_t n_piece = 0;
      int32_t t = 0, from = 0, to = 0;  // tile; blocks that some row sees
      bool more = true;
      const auto next_piece = [&] {
        more = get_piece(n_piece++, &piece);
        if (!more) return;
        t = piece.ta;
        to = (min(piece.pos0 + piece.positions, piece.len) - 1 >> shift) + 1;
        from = p.window > 0 ? max(max(piece.pos0, -1) - p.window + 1, 0) >> shift : 0;
      };
      next_piece();
      const auto ahead = [&](Ahead* a) {  // the next tile's table entry
        a->live = more;
        if (!more) return;
        a->head = piece.head;
        a->first = t == piece.ta;
        const int32_t j = (t * kTile + (lane & 7) * 16) >> shift;
        a->block = -1;
        if (lane < 8 && j < to && j >= from)
          a->block = __ldg(p.block_tables + piece.req * p.bt_stride + j);
        if (++t == piece.tb) next_piece();
      };
      const auto in_cache = [&](const Ahead& a) { return a.block >= 0 && a.block < p.num_blocks; };
      const auto scales_of = [&](const Ahead& a) {
        float2 s = make_float2(0.f, 0.f);
        if (a.live && lane < 8 && in_cache(a))
          s = __ldg(reinterpret_cast<const float2*>(p.kv + a.block * p.block_stride + a.head * p.head_stride +
                                                    (2 * D << shift)));
        return s;
      };
      Ahead a0, a1;
      ahead(&a0);
      float2 s0 = scales_of(a0);
      ahead(&a1);
      uint32_t j = 0, stage = 0, phase = 0;
      float ref = 0.f, most = 0.f;  // largest value scales: of the first tile that has one, of all so far
#pragma unroll 1
      while (a0.live) {
        const float2 s1 = scales_of(a1);
        Ahead a2;
        ahead(&a2);
        // Scales, by the lanes that have them; made before the stage is free (after the wait
        // they hold up the copies: 32 x 32768 decode 3 % slower).
        const bool here = lane < 8 && in_cache(a0);
        const bool zero = s0.y == 0.f, bad = !(s0.y >= 0.f && s0.y < INFINITY);
        const float own = here && !zero && !bad ? s0.y : 0.f;
        const uint32_t flags = __ballot_sync(kFull, here && zero) | __ballot_sync(kFull, here && bad) << 8 |
                               __ballot_sync(kFull, here) << 16 | __ballot_sync(kFull, here && s0.x < 0.f) << 24;
        if (a0.first) ref = most = 0.f;
        most = fmaxf(most, own);
        if (ref == 0.f || (flags & 0xFFFFu) != 0u) {  // (a tile without scales of zero needs the largest one at first only)
          most = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(most)));
          if (ref == 0.f) ref = most;  // (until a tile has values their scale is 0, like theirs)
        }
        float vlog = 0.f;
        if (own > 0.f)
          vlog = fminf(fmaxf(log2f(own / ref), kMinScaleLog), kMaxScaleLog);
        else if (here)
          vlog = (ref > 0.f ? fminf(log2f(most / ref), kMaxScaleLog) : 0.f) + kNoScaleLog;
        if (!wait(bar(L::kEmptyB, stage), phase ^ 1u, abort_flag, kSiteStageEmpty)) break;
        TileScales& sc = tile_scales[j % kScaleSlots];
        if (lane < 8) {
          sc.key[lane] = s0.x * p.scale_log2;
          sc.vlog[lane] = vlog;
          sc.vinv[lane] = ex2(-vlog);
          if (lane == 0) {
            sc.ref = ref;
            sc.flags = flags;
          }
        }
        __syncwarp();
        const bool leader = lane < 8 && (lane * 16 & ((1 << shift) - 1)) == 0;
        const int32_t block = here ? a0.block : p.num_blocks;  // (outside: zeros)
        const uint32_t rows = lane * 16 * 128u;
        if (lane == 0) {
          ptx::mbar_arrive(bar(L::scaleFullB, j % kScaleSlots));
          ptx::mbar_arrive_expect_tx(bar(L::kFullB, stage), L::kHalf);
        }
        __syncwarp();
        if (leader)
          ptx::tma_load_4d(base + L::k + stage * L::kHalf + rows, &tm_kv, bar(L::kFullB, stage), 0, 0, a0.head, block);
        if constexpr (D == 128) {
          if (!wait(bar(L::vEmptyB, stage), phase ^ 1u, abort_flag, kSiteStageEmpty)) {
            ++j;
            break;
          }
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar(L::vFullB, stage), L::kHalf);
          __syncwarp();
          if (leader)
            ptx::tma_load_4d(base + L::v + stage * L::kHalf + rows, &tm_kv, bar(L::vFullB, stage), D, 0, a0.head, block);
        }
        ++j;
        if (++stage == S) stage = 0, phase ^= 1u;
        a0 = a1;
        s0 = s1;
        a1 = a2;
      }
      __syncwarp();
      if (*abort_flag && lane == 0) {  // copies in flight must land before the memory is given back
        for (uint32_t i = j > S ? j - S : 0; i < j; ++i) {
          wait_drain(bar(L::kFullB, i % S), (i / S) & 1u, &g_block_attn_watchdog);
          if (D == 128) wait_drain(bar(L::vFullB, i % S), (i / S) & 1u, &g_block_attn_watchdog);
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // =========================== the products ===========================
      // One thread waits for and issues all of them.
      constexpr uint32_t kIdescS = ptx::idesc_e4m3_f32(128, kTile);
      constexpr uint32_t kIdescO = ptx::idesc_f16_f32(128, D) | ptx::kIdescMnMajorB;
      const uint64_t q0 = ptx::smem_desc_sw128(base + L::q), k0 = ptx::smem_desc_sw128(base + L::k);
      const uint64_t v0 = ptx::smem_desc_mn16(base + L::v16, kTile * 128u);
      if (ptx::elect_one()) {
        Ring ks{0u, 0u, static_cast<uint32_t>(S)}, vs{0u, 0u, static_cast<uint32_t>(kScaleSlots)}, us{0u, 0u, static_cast<uint32_t>(kUnitSlots)};
        uint32_t buf = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;  // f16 buffer; queries and probabilities of each group so far
        bool ok = true;
#pragma unroll 1
        while (true) {
          if (!wait_alone(bar(L::unitFullB, us.idx), us.phase, abort_flag, kSiteQEmpty)) break;
          const Piece& piece = *slot_of(us.idx);
          const int tiles = piece.tb - piece.ta;
          const bool shared = piece.shared != 0, last = piece.row0 < 0;
          ptx::mbar_arrive(bar(L::unitEmptyB, us.idx));
          us.next();
          if (last) break;
          const int count0 = shared ? tiles : (tiles + 1) / 2, count1 = shared ? tiles : tiles / 2;
          // Scores of group g's next tile; its tile's place is free after both groups' (its own) scores.
          const auto scores = [&](int g) {
            if ((!shared || g == 0) && !wait_alone(bar(L::kFullB, ks.idx), ks.phase, abort_flag, kSiteStageFull)) return false;
            ptx::tc_fence_after();
            const uint64_t a = q0 + static_cast<uint64_t>((shared ? g : 0) * (L::qBytes >> 4));
            const uint64_t b = k0 + static_cast<uint64_t>(ks.idx * (L::kHalf >> 4));
            const uint32_t d = tmem + g * kTile;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                ptx::mma_f8f6f4(d, a + part * (D == 128 ? L::kHalf >> 4 : 4u) + 2ull * kk, b + 2ull * kk, kIdescS,
                                part + kk > 0 ? 1u : 0u);
            ptx::mma_commit(bar(L::sFullB, g));
            if (!shared || g == 1) {
              ptx::mma_commit(bar(L::kEmptyB, ks.idx));
              ks.next();
            }
            return true;
          };
          // Outputs of group g's oldest tile, the i-th of n_g.
          const auto outputs = [&](int g, int i, int n_g) {
            if ((!shared || g == 0) && !wait_alone(bar(L::v16FullB, vs.idx), vs.phase, abort_flag, kSiteStageFull)) return false;
            if (!wait_alone(bar(L::pFullB, g), (g ? np1 : np0) & 1u, abort_flag, kSiteAccEmpty)) return false;
            if (g) ++np1; else ++np0;
            ptx::tc_fence_after();
            const uint64_t b = v0 + static_cast<uint64_t>(buf * (L::kV16 >> 4));
            const uint32_t d = tmem + 2 * kTile + g * 128, a = tmem + g * kTile;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              ptx::mma_f16_ts(d, a + 8 * kk, b + static_cast<uint64_t>(kk * (2048 >> 4)), kIdescO, i + kk > 0 ? 1u : 0u);
            if (!shared || g == 1) {
              ptx::mma_commit(bar(L::v16EmptyB, buf));
              buf ^= 1u;
              vs.next();
            }
            if (i + 1 == n_g) ptx::mma_commit(bar(L::oFullB, g));
            return true;
          };
          ok = wait_alone(bar(L::qFullB, 0), nq0 & 1u, abort_flag, kSiteQFull);
          ++nq0;
          if (ok && shared) {
            ok = wait_alone(bar(L::qFullB, 1), nq1 & 1u, abort_flag, kSiteQFull);
            ++nq1;
          }
          // A group's outputs of a tile, then its scores of the next.
#pragma unroll 1
          for (int i = -1; ok && i < count0; ++i) {
#pragma unroll 1
            for (int g = 0; ok && g < 2; ++g) {
              const int n_g = g ? count1 : count0;
              if (i >= 0 && i < n_g) ok = outputs(g, i, n_g);
              if (ok && i + 1 < n_g) ok = scores(g);
            }
          }
          if (!ok) break;
        }
        if (*abort_flag) {  // products in flight must end before the memory is given back
          ptx::mma_commit(bar(L::drainB));
          wait_drain(bar(L::drainB), 0, &g_block_attn_watchdog);
        }
      }
      __syncwarp();
    }
  } else if (warp >= kConvWarp0) {
    // ========================= values to f16 =========================
    reg_dec<kConvRegs>();
    const int w = warp - kConvWarp0;  // its 32 tokens of a tile
    const ConvPlace<D> at(w, lane);
    uint32_t j = 0, stage = 0, phase = 0;
    Piece piece;
    bool ok = true;
#pragma unroll 1
    for (uint32_t n = 0; ok && get_piece(n, &piece); ++n) {
#pragma unroll 1
      for (int t = piece.ta; t < piece.tb; ++t) {
        const uint32_t buf = j & 1u;
        ok = wait(bar(L::v16EmptyB, buf), ((j >> 1) & 1u) ^ 1u, abort_flag, kSiteAccFull) &&
             wait(bar(D == 128 ? L::vFullB : L::kFullB, stage), phase, abort_flag, kSiteStageFull);
        if (!ok) break;
        const uint32_t flags = tile_scales[j % kScaleSlots].flags;
        const uint8_t* const src = smem + L::v + stage * L::kHalf;
        uint8_t* const dst = smem + L::v16 + buf * L::kV16;
        uint32_t odd = flags & 0xFFFFu, nan_rows = 0;
        uint4 next[2] = {at.load(src, 0), at.load(src, 1)};
#pragma unroll 2
        for (int i = 0; i < ConvPlace<D>::kTimes; i += 2) {
          const uint4 codes[2] = {next[0], next[1]};
          if (i + 2 < ConvPlace<D>::kTimes) next[0] = at.load(src, i + 2), next[1] = at.load(src, i + 3);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // NaN codes (0x7F and 0xFF): adding one to the lower seven bits reaches the eighth
            odd |= ((codes[x].x & 0x7F7F7F7Fu) + 0x01010101u | (codes[x].y & 0x7F7F7F7Fu) + 0x01010101u |
                    (codes[x].z & 0x7F7F7F7Fu) + 0x01010101u | (codes[x].w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            at.store(dst, i + x, codes[x]);
          }
        }
        if (__any_sync(kFull, odd != 0u)) {
          nan_rows = convert_odd<D>(dst, src, w, lane, flags);
          if (nan_rows != 0u && lane == 0) *odd_values = 1u;
        }
        // the codes have been read: the stage may be filled again
        if (lane == 0) ptx::mbar_arrive(bar(D == 128 ? L::vEmptyB : L::kEmptyB, stage));
        if (lane == 0) reinterpret_cast<uint32_t*>(&tile_scales[j % kScaleSlots].nan)[w] = nan_rows;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::v16FullB, j % kScaleSlots));
        ++j;
        if (++stage == S) stage = 0, phase ^= 1u;
      }
    }
  } else {
    // ============================ the softmax ============================
    reg_inc<kSoftmaxRegs>();
    const int g = warp >> 2, quad = warp & 3;
    const int i = threadIdx.x & 127;  // lane of the accumulators
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_tm = tmem + g * kTile + lane_off, o_tm = tmem + 2 * kTile + g * 128 + lane_off;
    uint32_t j0 = 0, n_tiles = 0, n_outs = 0, n_meet = 0;
    const auto meet = [&] {  // the two groups
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(L::meetB));
      return wait(bar(L::meetB), n_meet++ & 1u, abort_flag, kSiteAccFull);
    };
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
      // (the piece stays in its slot: the registers are for the scores)
      if (!wait(bar(L::unitFullB, n % kUnitSlots), (n / kUnitSlots) & 1u, abort_flag, kSiteQEmpty)) goto out;
      const Piece& piece = *slot_of(n);
      if (piece.row0 < 0) break;
      const bool shared = piece.shared != 0;
      const int half = p.half_positions;
      // Lanes of a copy of the rows, and this thread's row.  (Two copies at least:
      // 350 us for 32 requests of 8 rows a key head, 17.0 for one of 4; one a
      // group: 376 and 17.7; four and eight, as here: 337 and 15.2.)
      const int rows = shared ? kTile : piece.positions * p.group;
      const int copy_lanes = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
      float row_scale;
      int pos = -1;
      {
        const int r = i & (copy_lanes - 1), index = r / p.group, h = r - index * p.group;  // position (of this group's), head
        const int position = index + (shared ? g * half : 0);
        const bool live = index < half && position < piece.positions;
        const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(p.q) +
                                       (static_cast<int64_t>(piece.row0) + position) * p.q_row_stride +
                                       (piece.head * p.group + h) * p.q_head_stride;
        const bool write = shared || g == 0;
        row_scale = load_query<D>(smem + L::q + g * L::qBytes, r, i / copy_lanes, kTile / copy_lanes, copy_lanes,
                                   live ? q : nullptr, write, p.negative ? 0x80000000u : 0u);
        if (write) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(L::qFullB, g));
        }
        if (live) pos = max(piece.pos0 + position, -1);
      }
      const int len = piece.len;
      const int full_to = min(piece.pos0 + 1, len);                  // positions below are seen by every row,
      const int full_from = p.window > 0 ? max(piece.pos0 + piece.positions - 1, -1) - p.window + 1 : 0;  // from here on
      const int chunk0 = quad / (copy_lanes / 32) * (copy_lanes / 32);
      const int step = shared ? 1 : 2, first = shared ? 0 : g;
      const int count = (piece.tb - piece.ta - first + step - 1) / step;
      RowState st;
      float ref = 0.f;
      uint32_t j = j0 + first;
      int tile0 = (piece.ta + first) * kTile;
      j0 += piece.tb - piece.ta;
      // Whether the row sees a NaN among the values of this group's last n tiles
      // before tile jj, which starts at `at`.  (Their scores' successors, which
      // this group has waited for, were issued after their products, and those
      // after their values had been converted: flag and masks are there.  They
      // stay until the third tile of the group after them is through.)
      const auto see_nan = [&](uint32_t jj, int at, int n) {
        if (*odd_values != 0u)
          st.bad |= sees_nan(tile_scales, jj, at, step, n, chunk0, chunk0 + copy_lanes / 32, pos, p.window, len);
      };
#pragma unroll 1
      for (int k = 0; k < count; ++k, j += step, tile0 += step * kTile) {
        if (!wait(bar(L::scaleFullB, j % kScaleSlots), (j / kScaleSlots) & 1u, abort_flag, kSiteStageFull) ||
            !wait(bar(L::sFullB, g), n_tiles & 1u, abort_flag, kSiteAccFull))
          goto out;
        ++n_tiles;
        ptx::tc_fence_after();
        {
          const TileScales& sc = tile_scales[j % kScaleSlots];
          ref = sc.ref;
          // (the flags: a block that is not there, a negative key scale)
          const bool masked = tile0 + kTile > full_to || tile0 < full_from || (sc.flags >> 16) != 0xFFu;
          softmax_tile<D>(s_tm, o_tm, sc, chunk0, copy_lanes / 32, masked, pos, p.window, len, tile0, row_scale, k == 0, st);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::pFullB, g));
        if ((k & 1) == 0 && k > 0) see_nan(j, tile0, 2);
      }
      if (count > 0) {
        if (!wait(bar(L::oFullB, g), n_outs & 1u, abort_flag, kSiteAccFull)) goto out;
        see_nan(j, tile0, (count & 1) != 0 ? 1 : 2);
        ++n_outs;
        ptx::tc_fence_after();
      }
      {
        // Where the results go: out, or the workspace.
        const int r = i & (copy_lanes - 1);
        float* const ws = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + piece.slot) * block_attn_piece_floats(D);
        if (shared) {
          const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
          const int index = r / p.group, position = index + g * half;
          const bool live = index < half && position < piece.positions;
          const int64_t row = static_cast<int64_t>(piece.row0) + position, head = piece.head * p.group + r - index * p.group;
          __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_row_stride + head * p.out_head_stride;
          const int wrow = g * kTile + i;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t a[32];
            ptx::tmem_ld_32x32b_x32(o_tm + c, a);
            ptx::tmem_wait_ld_regs(a);
            if (live) {
              if (st.bad) {
#pragma unroll
                for (int k = 0; k < 32; ++k) a[k] = 0x7FC00000u;
              }
              if (piece.slot < 0) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                  uint32_t w[4];
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    w[x] = bf16_pair(__uint_as_float(a[k + 2 * x]) * inv * ref, __uint_as_float(a[k + 2 * x + 1]) * inv * ref);
                  *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  __stcg(reinterpret_cast<uint4*>(ws + wrow * D + c + k), make_uint4(a[k], a[k + 1], a[k + 2], a[k + 3]));
              }
            }
            __syncwarp();  // (the next load is the whole warp's)
          }
          if (live) {
            if (piece.slot >= 0)
              __stcg(reinterpret_cast<float4*>(ws + kBlockAttnLanes * D) + wrow, make_float4(st.m, st.l, ref, 0.f));
            else if (p.lse)
              p.lse[row * p.heads + head] = st.l == 0.f ? -INFINITY : (st.m + log2f(st.l)) * 0.6931471805599453f;
          }
        } else {
          // The copies of a row meet: their maxima and sums first, then 32
          // channels at a time.
          float* const stage = reinterpret_cast<float*>(smem + L::q + L::qBytes);
          const int copies = 2 * kTile / copy_lanes, copy = (g * kTile + i) / copy_lanes;
          float4* const sums = reinterpret_cast<float4*>(stage);
          sums[g * kTile + i] = make_float4(st.m, st.l, ref, 0.f);
          if (!meet()) goto out;
          float m = kMinM, l = 0.f;
#pragma unroll 1
          for (int k = 0; k < copies; ++k) m = fmaxf(m, sums[k * copy_lanes + r].x);
#pragma unroll 1
          for (int k = 0; k < copies; ++k) {
            const float4 v = sums[k * copy_lanes + r];
            l = fmaf(v.y, ex2(v.x - m), l);
          }
          ref = fmaxf(sums[0].z, sums[kTile].z);  // (0 before the first tile with values)
          const float f = ex2(st.m - m);
          // A round takes as many channels as 32 KB hold of all copies' rows in use,
          // and a thread puts out `share` of them for one row.
          const int pad = D == 128 && rows <= 8 ? 8 : rows <= 16 ? 16 : copy_lanes;  // (at most D channels)
          const int width = 32 * copy_lanes / pad, share = copy_lanes / 8, tid = threadIdx.x;
          const int to_row = tid / (256 / pad), to_col = tid % (256 / pad) * share;
          const int to_index = to_row / p.group, to_head = piece.head * p.group + to_row - to_index * p.group;
          const bool to_live = to_row < rows;
          // (the row that this thread puts out is another one than its own: its sum through the stage)
          if (!meet()) goto out;
          if (copy == 0) sums[r] = make_float4(m, l, ref, 0.f);
          if (!meet()) goto out;
          const float4 to_ml = sums[to_row];
          const float inv = to_ml.y == 0.f ? 0.f : 1.f / to_ml.y;
          const int64_t out_row = static_cast<int64_t>(piece.row0) + to_index;
          __nv_bfloat16* const out =
              static_cast<__nv_bfloat16*>(p.out) + out_row * p.out_row_stride + to_head * p.out_head_stride;
          if (to_live && to_col == 0) {
            if (piece.slot >= 0)
              __stcg(reinterpret_cast<float4*>(ws + kBlockAttnLanes * D) + to_row, make_float4(to_ml.x, to_ml.y, ref, 0.f));
            else if (p.lse)
              p.lse[out_row * p.heads + to_head] =
                  to_ml.y == 0.f ? -INFINITY : (to_ml.x + log2f(to_ml.y)) * 0.6931471805599453f;
          }
#pragma unroll 1
          for (int c = 0; c < D; c += width) {
            if (!meet()) goto out;  // (what stood there has been read)
#pragma unroll 1
            for (int x = 0; x < width; x += 32) {
              uint32_t a[32];
              if (count > 0) {
                ptx::tmem_ld_32x32b_x32(o_tm + c + x, a);
                ptx::tmem_wait_ld_regs(a);
              }
              if (r < pad) {
                float* const mine = stage + (copy * pad + r) * width + x;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (count > 0)
                    v = make_float4(__uint_as_float(a[4 * k]) * f, __uint_as_float(a[4 * k + 1]) * f,
                                    __uint_as_float(a[4 * k + 2]) * f, __uint_as_float(a[4 * k + 3]) * f);
                  if (st.bad) v = make_float4(NAN, NAN, NAN, NAN);
                  *reinterpret_cast<float4*>(mine + ((k ^ (r & 7)) << 2)) = v;
                }
              }
              __syncwarp();  // (the next load is the whole warp's)
            }
            if (!meet()) goto out;
            if (to_live) {
#pragma unroll 1
              for (int x = to_col; x < to_col + share; x += 4) {
                const float* const from = stage + to_row * width + (x & ~31) + (((x >> 2 & 7) ^ (to_row & 7)) << 2);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int k = 0; k < copies; ++k) {
                  const float4 v = *reinterpret_cast<const float4*>(from + k * pad * width);
                  sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
                if (piece.slot >= 0)
                  __stcg(reinterpret_cast<float4*>(ws + to_row * D + c + x), sum);
                else
                  *reinterpret_cast<uint2*>(out + c + x) =
                      make_uint2(bf16_pair(sum.x * inv * ref, sum.y * inv * ref), bf16_pair(sum.z * inv * ref, sum.w * inv * ref));
              }
            }
          }
          if (!meet()) goto out;  // (group 1's queries may come where the copies met)
        }
        // the accumulator is read before the next piece's products overwrite it
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::unitEmptyB, n % kUnitSlots));
      }
    }
  out:;
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the units that several CTAs shared, in their order: a warp
// a row.  (Four rows a warp take 18 us where this takes 15 for one token, and
// save 1 us of 39 where every unit of 252 rows is cut.)
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) block_attn_join_kernel(const BlockAttnParams p) {
  const BlockAttnMeta meta = p.meta[blockIdx.x];
  if (meta.positions == 0) return;
  const int lane = threadIdx.x & 31, half = p.half_positions;
  constexpr int kPer = D / 32;
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), g = meta.shared ? r / kTile : 0;
  const int index = (r - g * kTile) / p.group, position = index + g * half;
  if ((meta.shared && index >= half) || position >= meta.positions) return;
  // (a record that another call in flight wrote into the same workspace leads nowhere else)
  const int last = min(meta.last, static_cast<int>(gridDim.x) - 1);
  const int head = meta.head * p.group + (r - g * kTile) - index * p.group;
  if (meta.row0 + position >= p.rows || head >= p.heads) return;
  // Outputs go by the power of two below the first value scale: their sums may be 2^15 times the mean.
  float top = kMinM, l = 0.f, over = 0.f, o[kPer] = {};
#pragma unroll 4
  for (int c = blockIdx.x; c <= last; ++c) {
    const float* const ws =
        p.partial + (static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x) ? 1 : 0)) * block_attn_piece_floats(D);
    const float4 ml = __ldcg(reinterpret_cast<const float4*>(ws + kBlockAttnLanes * D) + r);
    float2 v[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) v[i] = __ldcg(reinterpret_cast<const float2*>(ws + r * D + lane * kPer) + i);
    const float now = fmaxf(top, ml.x), f = ex2(top - now), e = ex2(ml.x - now);
    l = fmaf(ml.y, e, l * f);
    top = now;
    if (over == 0.f && ml.z > 0.f)  // (0: a piece without values)
      over = power_of_two(127 - min(max(static_cast<int>(__float_as_uint(ml.z) >> 23), 1), 253));
    const float by = e * (ml.z * over);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      o[2 * i] = fmaf(v[i].x, by, o[2 * i] * f);
      o[2 * i + 1] = fmaf(v[i].y, by, o[2 * i + 1] * f);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l, under = over > 0.f ? 1.f / over : 0.f;
  const int64_t row = static_cast<int64_t>(meta.row0) + position;
  __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_row_stride + head * p.out_head_stride;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(out + lane * kPer + i) = bf16_pair(o[i] * inv * under, o[i + 1] * inv * under);
  if (p.lse && lane == 0)
    p.lse[row * p.heads + head] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

namespace {
template <int D>
cudaError_t launch(const CUtensorMap& tm, const BlockAttnParams& p, int grid, cudaStream_t stream) {
  const int smem = static_cast<int>(Smem<D>::total);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(block_attn_kernel<D>), smem);
  if (e != cudaSuccess) return e;
  block_attn_kernel<D><<<grid, kThreads, smem, stream>>>(tm, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = p.rows <= p.half_positions ? p.rows * p.group : kBlockAttnLanes;  // (lanes of a second tile start at 128)
  block_attn_join_kernel<D><<<dim3(grid, (rows + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, stream>>>(p);
  return cudaGetLastError();
}
}  // namespace

int block_attn_smem(int head_dim) { return static_cast<int>(head_dim == 128 ? Smem<128>::total : Smem<64>::total); }

cudaError_t launch_block_attn(const CUtensorMap& tm, const BlockAttnParams& p, int head_dim, int grid, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(tm, p, grid, stream) : launch<64>(tm, p, grid, stream);
}

cudaError_t read_block_attn_watchdog(unsigned int* value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_block_attn_watchdog, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_block_attn_watchdog, &zero, sizeof(unsigned int));
}

}  // namespace fp8idx
