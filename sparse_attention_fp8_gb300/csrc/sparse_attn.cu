// Attention over the selected positions of a paged e4m3 key/value cache
// (fp8_paged_sparse_attn, fp8_mqa_sparse_attn_paged) for sm_103a.
//
//   s[h, j] = softmax_scale * <q[h], K[i_j]>,  out[h] = sum_j softmax(s)[h, j] V[i_j]
//
// A unit of work is (row, key head, up to 64 of its query heads); its entries
// are taken in tiles of 128 tokens.  Both products of a tile run on the fp8
// tensor cores straight from the cache's bytes:
//   S^T [128 tokens x 2 GP] = K tile (A, K-major) * [Qh; Ql]^T
//   O^T [128 channels x 2 GP] += V tile^T (A, MN-major) * [Ph | Pl] (B, MN-major)
// GP is the head count padded to 16, 32 or 64.  The 16-bit operands are split
// into two e4m3 values: x = h + l / 16 with h = e4m3(x), l = e4m3(16 (x - h)).
// That keeps 8 significant bits -- a bf16 query exactly, a probability to
// 2^-8 -- down to 2^-21 of the largest query element (queries are scaled by a
// power of two so that it lies in [128, 256)).  The two halves have their own
// accumulator columns and meet in f32.  Dequantising the tile to 16 bits
// instead would take a conversion per cache byte and twice the shared memory.
//
// The gather bounds this kernel: a unit reads 2*D + 8 bytes per entry, once
// per row and key head, mostly from L2, while the two products need little
// (with 32 heads a tile's eight MMAs take about a third of its copy).  So a
// unit's tile is M = 128 tokens by all heads of the key head, every byte is
// fetched once, and a ring of tiles keeps the copies of several tiles in
// flight.
//
// Roles of a CTA (12 warps; persistent over units, or one unit per cluster):
//  * Producer warps (two, alternate tiles): each lane resolves four entries
//    to cache rows (block-table entries loaded one tile ahead, indices two)
//    and fetches their key and value rows with gathering TMA copies of four
//    rows, their scales with 8-byte cp.async.  Entries that select nothing
//    read row -1, which the copy fills with zeros; a tile without any entry
//    is published empty and costs no copy and no MMA.
//  * Query warp: splits the next unit's query into Qh and Ql.
//  * MMA warp: issues S of a later tile whenever its data is there, else the
//    output MMA of the oldest tile whose probabilities are.
//  * Epilogue warpgroups (two, alternate tiles; thread = token): scores times
//    the token's scale, probability 2^(t - m), its sum per head in the
//    thread, and P (scaled by the token's value scale) into shared memory as
//    the next MMA's operand.  Each group keeps its own maximum m, sums and
//    output accumulator, so the groups meet once per unit.
//    m is the maximum of the tile in which it was last set: a later tile that
//    stays below m + 2 (in log2) keeps it, so a tile needs one vote of the
//    group instead of a maximum per head across its 128 threads; a tile that
//    does not takes the exact maxima and rescales the sums and the
//    accumulator.  P then is at most 8 (4 for the score, 2 for the value
//    scale, kept the same way), 256 after the factor 32.
//  * Few units: a cluster of 2, 4 or 8 CTAs per unit, each with a share of
//    the tiles; their outputs meet in f32 through distributed shared memory.
// Every wait is bounded (common.cuh).  After a wait has run out the group
// votes, so that its four warps leave together and no barrier is left open.
#include <cooperative_groups.h>
#include <cuda.h>
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

constexpr int kProdWarp0 = 4 * kAttnGroups;
constexpr int kProdWarps = 2;
constexpr int kMmaWarp = kProdWarp0 + kProdWarps;
constexpr int kQWarp = kMmaWarp + 1;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLazy = 2.f;          // log2 of how far a score may pass m before m is set anew
constexpr float kPScale = 32.f;       // factor of P's e4m3 codes
constexpr float kMinVScale = 0x1p-120f;
constexpr float kMinM = -3e38f;       // m stays finite, so that a score of -inf gives probability 0

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Floats ordered as signed integers (NaN above all), and back.
__device__ __forceinline__ int float_key(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float key_float(int k) { return __int_as_float(k >= 0 ? k : k ^ 0x7FFFFFFF); }

// Softmax state of a CTA in shared memory.
template <int GP>
struct AttnState {
  float nm[2][GP];            // -m of each group (log2 units)
  float ninf[GP];             // -inf: the row of -m that an entry without a token reads
  float lred[2][2][4][GP];    // [unit parity][group][warp]: sums of the probabilities
  float msave[2][2][GP];      // [unit parity][group]: m at the unit's end
  float wmax[2][4][GP];       // [group][warp]: a tile's maxima
  float resc[2][GP];          // [group]: factor of a new maximum
  float fac[GP][2];           // factors of the groups' accumulators
  float xm[GP], xl[GP];       // cluster: this CTA's maximum and sum per head
  float csave[2][2];          // [unit parity][group]: the value scale that P is relative to
  float used[2][2];           // [unit parity][group]: 1 if its accumulator holds anything
  float cref[2], cfac[2];
  float wvs[2][4];
  float qf[2];                // [query buffer]: 2^-e of the query's scaling
};

struct Cursor {  // tiles [t0, t1) of units u, u + step, ...
  int u, t, t0, t1, step;
  __device__ __forceinline__ bool advance() {  // true: a new unit
    if (++t < t1) return false;
    t = t0;
    u += step;
    return true;
  }
};

struct Entries {  // a lane's four entries of a tile
  int32_t idx[4];
  int row, kvh;
};

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

}  // namespace

template <int D, int GP, bool CLUSTER>
__global__ void __launch_bounds__(kAttnThreads, 1)
    sparse_attn_kernel(const __grid_constant__ CUtensorMap tm_kv, const SparseAttnParams p) {
  constexpr int N2 = 2 * GP;                       // columns of S^T and O^T
  constexpr uint32_t kStageBytes = kAttnTile * 2u * D;
  constexpr uint32_t kVOff = D == 128 ? kAttnTile * 128u : 0u;  // D = 64: key and value share a 128-byte row
  constexpr uint32_t kTmemCols = 4u * N2;          // S and O of two groups
  static_assert(sizeof(AttnState<GP>) <= 4u * attn_state_floats(GP), "state");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_1024(smem_raw);
  const AttnSmem L = attn_smem_layout(D, GP, p.stages);
  const int S = p.stages;
  AttnState<GP>& stt = *reinterpret_cast<AttnState<GP>*>(smem + L.flt);
  const uint32_t kv0 = ptx::smem_u32(smem + L.kv);
  const uint32_t q0 = ptx::smem_u32(smem + L.q);
  const uint32_t bars = ptx::smem_u32(smem + L.bars);
  const uint32_t full0 = bars, empty0 = full0 + 8u * kAttnMaxStages;
  const uint32_t qf0 = empty0 + 8u * kAttnMaxStages, qe0 = qf0 + 16u;  // query buffers
  const uint32_t sf0 = qe0 + 16u, se0 = sf0 + 16u;  // [group] scores ready, read
  const uint32_t pf0 = se0 + 16u, pe0 = pf0 + 16u;  // [group] probabilities ready, used
  const uint32_t ub = pe0 + 16u, oe = ub + 8u;      // unit ends: both groups done; accumulators read
  const uint32_t drain_bar = oe + 8u;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L.misc);
  volatile uint32_t* abort_flag = misc + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    misc[1] = 0u;
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full0 + 8u * s, 32u + 1u);  // the producer lanes' scale copies, the copies' bytes
      ptx::mbar_init(empty0 + 8u * s, 1u + 4u);  // the output MMA, the tile's epilogue warps
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(qf0 + 8u * g, 1u);
      ptx::mbar_init(qe0 + 8u * g, 1u + 4u * kAttnGroups);
      ptx::mbar_init(sf0 + 8u * g, 1u);
      ptx::mbar_init(se0 + 8u * g, 4u);
      ptx::mbar_init(pf0 + 8u * g, 4u);
      ptx::mbar_init(pe0 + 8u * g, 1u);
    }
    ptx::mbar_init(ub, 4u * kAttnGroups);
    ptx::mbar_init(oe, 4u * kAttnGroups);
    ptx::mbar_init(drain_bar, 1u);
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tm_kv);
  }
  for (int g = threadIdx.x; g < GP; g += kAttnThreads) stt.ninf[g] = -INFINITY;
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(misc), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  // this CTA's units and tiles
  const int C = CLUSTER ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
  const int crank = CLUSTER ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int per = (p.tiles + C - 1) / C;
  const int t0 = min(crank * per, p.tiles), t1 = min(t0 + per, p.tiles);
  const int u0 = CLUSTER ? static_cast<int>(blockIdx.x) / C : static_cast<int>(blockIdx.x);
  const int ustep = CLUSTER ? p.units : static_cast<int>(gridDim.x);
  const int n_units = u0 < p.units ? (p.units - u0 + ustep - 1) / ustep : 0;
  const int total = n_units * (t1 - t0);

  if (warp >= kProdWarp0 && warp < kProdWarp0 + kProdWarps) {
    // ============================ producers ============================
    const int pw = warp - kProdWarp0;
    const int bs = p.block_size, shift = p.block_shift;
    const auto load_entries = [&](const Cursor& c, Entries& en) {
      int h0;
      unit_of(p, c.u, &en.row, &en.kvh, &h0, GP);
      const int at = c.t * kAttnTile + 4 * lane;
      const int32_t* src = p.indices + en.row * p.idx_stride + at;
      if (p.idx_vec && at + 3 < p.k) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(src));
        en.idx[0] = v.x, en.idx[1] = v.y, en.idx[2] = v.z, en.idx[3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) en.idx[i] = at + i < p.k ? __ldg(src + i) : -1;
      }
    };
    // block-table entries (or -1) and places in the page of four entries
    int req_guess = 0;
    const auto load_tables = [&](const Entries& en, int32_t (&blk)[4], int (&off)[4]) {
      const int req_row = en.row / p.next_n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int32_t tok = en.idx[i];
        int req = req_row;
        bool ok = tok >= 0;
        if (p.cu_seq_lens != nullptr && ok) {
          // the request of a column: the last one found, or a search
          int32_t lo = __ldg(p.cu_seq_lens + req_guess), hi = __ldg(p.cu_seq_lens + req_guess + 1);
          if (tok < lo || tok >= hi) {
            int a = 0, b = p.n_req;
            while (b - a > 1) {
              const int mid = (a + b) >> 1;
              if (__ldg(p.cu_seq_lens + mid) <= tok) a = mid; else b = mid;
            }
            req_guess = a;
            lo = __ldg(p.cu_seq_lens + a);
            hi = __ldg(p.cu_seq_lens + a + 1);
          }
          ok = tok >= lo && tok < hi;
          req = req_guess;
          tok -= lo;
        }
        const int32_t j = tok >> shift;
        off[i] = tok & (bs - 1);
        blk[i] = ok && j < p.max_blocks ? __ldg(p.block_tables + req * p.bt_stride + j) : -1;
      }
    };
    Cursor cur{u0, t0, t0, t1, ustep};
    Ring st{0u, 0u, static_cast<uint32_t>(S)};
    if (pw < total) {
      // walk to this warp's first tile, and one of its tiles further for each look-ahead
      const auto next_own = [&](Cursor& c) {
        for (int i = 0; i < kProdWarps; ++i) c.advance();
      };
      for (int i = 0; i < pw; ++i) {
        cur.advance();
        st.next();
      }
      Entries en, en1, en2;
      int32_t blk[4], blk1[4];
      int off[4], off1[4];
      Cursor ahead = cur;
      load_entries(ahead, en);
      load_tables(en, blk, off);
      next_own(ahead);
      if (pw + kProdWarps < total) load_entries(ahead, en1);
      int issued = 0;
      bool okay = true;
      for (int it = pw; it < total && okay; it += kProdWarps) {
        if (it + kProdWarps < total) load_tables(en1, blk1, off1);
        next_own(ahead);
        if (it + 2 * kProdWarps < total) load_entries(ahead, en2);
        uint32_t own = 0;
        int32_t row[4];
        const uint8_t* sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool ok = blk[i] >= 0 && blk[i] < p.num_blocks;
          own |= (ok ? 1u : 0u) << i;
          row[i] = ok ? static_cast<int32_t>(blk[i] * p.row_block + en.kvh * p.row_head +
                                             static_cast<int64_t>(off[i]) * p.row_tok)
                      : -1;
          sc[i] = p.kv + blk[i] * p.block_stride + en.kvh * p.kv_head_stride + static_cast<int64_t>(bs) * 2 * D + 8 * off[i];
        }
        // tokens 32w .. 32w+31 are the entries of lanes 8w .. 8w+7
        uint32_t m = own << (4 * (lane & 7));
        m |= __shfl_xor_sync(kFull, m, 1);
        m |= __shfl_xor_sync(kFull, m, 2);
        m |= __shfl_xor_sync(kFull, m, 4);
        const bool any = __any_sync(kFull, m != 0u);
        okay = warp_wait_bounded(empty0 + 8u * st.idx, st.phase ^ 1u, abort_flag, &g_attn_watchdog, kSiteStageEmpty);
        if (!okay) break;
        if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(smem + L.mask)[4 * st.idx + (lane >> 3)] = m;
        const uint32_t full = full0 + 8u * st.idx;
        __syncwarp();
        if (lane == 0) {
          if (any)
            ptx::mbar_arrive_expect_tx(full, kStageBytes);
          else
            ptx::mbar_arrive(full);
        }
        __syncwarp();
        if (any) {
          const uint32_t dst = kv0 + st.idx * kStageBytes + lane * 4u * 128u;
          ptx::tma_gather4(dst, &tm_kv, full, 0, row[0], row[1], row[2], row[3]);
          if constexpr (D == 128) {
            const int dy = p.v_dy;
            ptx::tma_gather4(dst + kVOff, &tm_kv, full, p.v_dx, row[0] < 0 ? -1 : row[0] + dy,
                             row[1] < 0 ? -1 : row[1] + dy, row[2] < 0 ? -1 : row[2] + dy,
                             row[3] < 0 ? -1 : row[3] + dy);
          }
          const uint32_t sdst = ptx::smem_u32(smem + L.scale) + (st.idx * kAttnTile + 4u * lane) * 8u;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (own >> i & 1u) ptx::cp_async_8(sdst + 8u * i, sc[i]);
        }
        ptx::cp_async_mbar_arrive(full);
        issued = it + 1;
        for (int i = 0; i < kProdWarps; ++i) st.next();
        en = en1;
        en1 = en2;
#pragma unroll
        for (int i = 0; i < 4; ++i) blk[i] = blk1[i], off[i] = off1[i];
      }
      if (*abort_flag && lane == 0)  // let issued copies land before the CTA exits
        for (int it = max(0, issued - S); it < issued; ++it)
          if (it % kProdWarps == pw) wait_drain(full0 + 8u * (it % S), (it / S) & 1, &g_attn_watchdog);
    }
  } else if (warp == kQWarp) {
    // ============================ queries ==============================
    uint32_t phase = 0;
    if (total > 0) {
      for (int i = 0; i < n_units; ++i) {
        const int buf = i & 1;
        int row, kvh, h0;
        unit_of(p, u0 + i * ustep, &row, &kvh, &h0, GP);
        const int nh = min(GP, p.group - h0);
        if (!warp_wait_bounded(qe0 + 8u * buf, ((phase >> buf) & 1u) ^ 1u, abort_flag, &g_attn_watchdog, kSiteQEmpty))
          break;
        phase ^= 1u << buf;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row / p.next_n * p.q_req_stride +
                                 row % p.next_n * p.q_row_stride + (kvh * p.group + h0) * p.q_head_stride;
        constexpr int kPer = D / 8;  // 16-byte pieces per head
        float amax = 0.f;
#pragma unroll 4
        for (int c = lane; c < nh * kPer; c += 32) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + c / kPer * p.q_head_stride + c % kPer * 8));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = fabsf(__uint_as_float(w[k] << 16)), b = fabsf(__uint_as_float(w[k] & 0xFFFF0000u));
            if (a < INFINITY) amax = fmaxf(amax, a);
            if (b < INFINITY) amax = fmaxf(amax, b);
          }
        }
        amax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(amax)));
        // 2^e puts the largest finite element into [128, 256)
        int e = 134 - static_cast<int>(__float_as_uint(amax) >> 23);
        e = amax == 0.f ? 0 : min(max(e, -120), 120);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        uint8_t* dst = smem + L.q + buf * N2 * 128;
#pragma unroll 4
        for (int c = lane; c < GP * kPer; c += 32) {
          const int g = c / kPer, piece = c % kPer;
          uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
          if (g < nh) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + g * p.q_head_stride + piece * 8));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a = __uint_as_float(w[k] << 16) * mul, b = __uint_as_float(w[k] & 0xFFFF0000u) * mul;
              if (isinf(a)) a = NAN;  // (an infinity must not become the largest code)
              if (isinf(b)) b = NAN;
              const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
              const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
              const __nv_fp8x2_storage_t l = __nv_cvt_float2_to_fp8x2(
                  make_float2(16.f * (a - back.x), 16.f * (b - back.y)), __NV_SATFINITE, __NV_E4M3);
              hi[k >> 1] |= static_cast<uint32_t>(h) << (16 * (k & 1));
              lo[k >> 1] |= static_cast<uint32_t>(l) << (16 * (k & 1));
            }
          }
          // rows of 128 bytes in the 128-byte swizzle (16-byte chunks)
          const int chunk = piece >> 1, half = (piece & 1) * 8;
          const int r1 = g, r2 = GP + g;
          *reinterpret_cast<uint2*>(dst + r1 * 128 + ((chunk ^ (r1 & 7)) << 4) + half) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(dst + r2 * 128 + ((chunk ^ (r2 & 7)) << 4) + half) = make_uint2(lo[0], lo[1]);
        }
        if (lane == 0) stt.qf[buf] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(qf0 + 8u * buf);
      }
    }
  } else if (warp == kMmaWarp) {
    // ============================== MMA ================================
    if (lane == 0 && total > 0) {
      constexpr uint32_t kIdescS = ptx::idesc_e4m3_f32(kAttnTile, N2);
      constexpr uint32_t kIdescO = ptx::idesc_e4m3_f32(128, N2) | ptx::kIdescMnMajorA | ptx::kIdescMnMajorB;
      const uint64_t q_desc = ptx::smem_desc_sw128(q0);
      const uint32_t p0 = ptx::smem_u32(smem + L.p);
      Cursor cs{u0, t0, t0, t1, ustep}, cp = cs;     // tiles whose scores, outputs come next
      Ring rs{0u, 0u, static_cast<uint32_t>(S)}, rp = rs;
      int is = 0, ip = 0, us = 0, up = 0;             // tile and unit counts
      uint32_t ns = 0, np = 0;                        // bit g: parity of the tiles of group g
      uint32_t started = 0;                           // bit g: its accumulator holds this unit's sums
      const auto tile_any = [&](uint32_t stage) {
        const uint4 m = *reinterpret_cast<const uint4*>(smem + L.mask + 16 * stage);
        return (m.x | m.y | m.z | m.w) != 0u;
      };
      uint64_t since = 0;
      uint32_t spins = 0;
      while (ip < total) {
        bool did = false;
        if (is < total && ptx::mbar_test_wait(full0 + 8u * rs.idx, rs.phase)) {
          const uint32_t g = is & 1;
          const bool any = tile_any(rs.idx);
          if (!any || (ptx::mbar_test_wait(qf0 + 8u * (us & 1), (us >> 1) & 1) &&
                       ptx::mbar_test_wait(se0 + 8u * g, ((ns >> g) & 1u) ^ 1u))) {
            if (any) {
              ptx::tc_fence_after();
              const uint64_t a = ptx::smem_desc_sw128(kv0 + rs.idx * kStageBytes);
              const uint64_t b = q_desc + ((us & 1) * N2 * 128u >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                ptx::mma_f8f6f4(tmem + g * N2, a + 2ull * kk, b + 2ull * kk, kIdescS, kk > 0 ? 1u : 0u);
              ptx::mma_commit(sf0 + 8u * g);
              ns ^= 1u << g;
            }
            ++is;
            rs.next();
            if (cs.advance()) {
              ptx::mma_commit(qe0 + 8u * (us & 1));
              ++us;
            }
            did = true;
          }
        }
        if (!did && ip < is) {
          const uint32_t g = ip & 1;
          const bool any = tile_any(rp.idx);
          const bool first = !(started >> g & 1u);
          if (!any || (ptx::mbar_test_wait(pf0 + 8u * g, (np >> g) & 1u) &&
                       (!first || up == 0 || ptx::mbar_test_wait(oe, (up - 1) & 1)))) {
            if (any) {
              ptx::tc_fence_after();
              const uint64_t a = ptx::smem_desc_mn(kv0 + rp.idx * kStageBytes + kVOff, 128);
              const uint64_t b = ptx::smem_desc_mn(p0 + g * kAttnTile * N2, N2);
#pragma unroll
              for (int kk = 0; kk < kAttnTile / 32; ++kk)
                ptx::mma_f8f6f4(tmem + (2 + g) * N2, a + kk * (32ull * 128 >> 4), b + kk * (32ull * N2 >> 4), kIdescO,
                                (first && kk == 0) ? 0u : 1u);
              ptx::mma_commit(pe0 + 8u * g);
              ptx::mma_commit(empty0 + 8u * rp.idx);
              np ^= 1u << g;
              started |= 1u << g;
            } else {
              ptx::mbar_arrive(empty0 + 8u * rp.idx);
            }
            ++ip;
            rp.next();
            if (cp.advance()) {
              ++up;
              started = 0;
            }
            did = true;
          }
        }
        if (did) {
          spins = 0;
        } else if ((++spins & 255u) == 0u) {
          if (*abort_flag) break;
          const uint64_t now = ptx::globaltimer_ns();
          if (spins == 256u) {
            since = now;
          } else if (now - since > kWaitTimeoutNs) {
            *abort_flag = 1u;
            atomicOr(&g_attn_watchdog, static_cast<uint32_t>(kSiteAccEmpty));
            break;
          }
        }
      }
      if (*abort_flag) {
        ptx::mma_commit(drain_bar);
        wait_drain(drain_bar, 0, &g_attn_watchdog);
      }
    }
  } else {
    // ============================ epilogue =============================
    const int g = warp >> 2, quad = warp & 3;
    const int tg = threadIdx.x & 127;                 // thread in the group = token = channel
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_tm = tmem + g * N2 + lane_off, o_tm = tmem + (2 + g) * N2 + lane_off;
    uint8_t* p_row = smem + L.p + g * kAttnTile * N2 + tg * N2;
    // 16-byte chunks of a row of probabilities, swizzled over its N2 bytes
    const uint32_t p_swz = N2 == 128 ? tg & 7 : N2 == 64 ? (tg >> 1) & 3 : (tg >> 2) & 1;
    const int bar_id = 1 + g;
    Ring st{0u, 0u, static_cast<uint32_t>(S)};
    uint32_t n_tile = 0;                              // this group's tiles so far
    int it = 0;
    bool stop = false;
    for (int i = 0; i < n_units && !stop; ++i) {
      const int buf = i & 1, par = i & 1;
      float qscale = 0.f;
      bool ok = true;
      if (total > 0) {
        ok = warp_wait_bounded(qf0 + 8u * buf, (i >> 1) & 1, abort_flag, &g_attn_watchdog, kSiteQFull);
        qscale = stt.qf[buf] * p.scale_log2;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(qe0 + 8u * buf);
      }
      bool has_o = false;
      float cref = 0.f;
      float2 l2[GP / 2];
#pragma unroll
      for (int j = 0; j < GP / 2; ++j) l2[j] = make_float2(0.f, 0.f);

      for (int t = t0; t < t1; ++t, ++it) {
        const uint32_t stage = st.idx, stage_phase = st.phase;
        st.next();
        if ((it & 1) != g) continue;
        ok = warp_wait_bounded(full0 + 8u * stage, stage_phase, abort_flag, &g_attn_watchdog, kSiteStageFull) && ok;
        const uint4 mk = *reinterpret_cast<const uint4*>(smem + L.mask + 16 * stage);
        const bool any = (mk.x | mk.y | mk.z | mk.w) != 0u;
        const uint32_t mw = quad == 0 ? mk.x : quad == 1 ? mk.y : quad == 2 ? mk.z : mk.w;
        const bool valid = mw >> lane & 1u;
        const float2 sc = reinterpret_cast<const float2*>(smem + L.scale)[stage * kAttnTile + tg];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty0 + 8u * stage);
        const float c = valid ? sc.x * qscale : 0.f;
        const float vs = valid ? fmaxf(sc.y, 0.f) : 0.f;
        const float4* nm4 = reinterpret_cast<const float4*>(valid ? stt.nm[g] : stt.ninf);
        const float2 c2 = make_float2(c, c), k16 = make_float2(0.0625f, 0.0625f);
        bool again = !has_o;  // the group's first tile of a unit sets m
        if (any) {
          ok = warp_wait_bounded(sf0 + 8u * g, n_tile & 1u, abort_flag, &g_attn_watchdog, kSiteAccFull) && ok;
          ptx::tc_fence_after();
          if (!again) {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < GP; b += 16) {
              uint32_t hi[16], lo[16];
              ptx::tmem_ld_32x32b_x16(s_tm + b, hi);
              ptx::tmem_ld_32x32b_x16(s_tm + GP + b, lo);
              ptx::tmem_wait_ld_n(hi);
              ptx::tmem_wait_ld_n(lo);
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 nm = nm4[(b + j) / 4];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const float2 raw = __ffma2_rn(make_float2(__uint_as_float(lo[j + k]), __uint_as_float(lo[j + k + 1])),
                                                k16,
                                                make_float2(__uint_as_float(hi[j + k]), __uint_as_float(hi[j + k + 1])));
                  const float2 t2 = __ffma2_rn(raw, c2, k == 0 ? make_float2(nm.x, nm.y) : make_float2(nm.z, nm.w));
                  top = fmaxf(top, fmaxf(t2.x, t2.y));
                }
              }
            }
            again = top > kLazy || vs > 2.f * cref;
          }
        }
        if (!any) again = false;
        if (ptx::bar_or(bar_id, 128, again || !ok)) {
          // ---- new maxima (or the end of an abandoned call)
          if (ptx::bar_or(bar_id, 128, !ok)) {
            stop = true;
            break;
          }
#pragma unroll 1
          for (int b = 0; b < GP; b += 16) {
            uint32_t hi[16], lo[16];
            ptx::tmem_ld_32x32b_x16(s_tm + b, hi);
            ptx::tmem_ld_32x32b_x16(s_tm + GP + b, lo);
            ptx::tmem_wait_ld_n(hi);
            ptx::tmem_wait_ld_n(lo);
            int mine = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float s = fmaf(__uint_as_float(lo[j]), 0.0625f, __uint_as_float(hi[j])) * c;
              const int m = __reduce_max_sync(kFull, float_key(valid ? s : -INFINITY));
              if (lane == j) mine = m;
            }
            if (lane < 16) stt.wmax[g][quad][b + lane] = key_float(mine);
          }
          const float vmax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vs)));
          if (lane == 0) stt.wvs[g][quad] = vmax;
          ptx::bar_sync(bar_id, 128);
          if (tg < GP) {
            const float old = has_o ? -stt.nm[g][tg] : kMinM;
            float m = old;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float x = stt.wmax[g][w][tg];
              m = (x > m || x != x) ? x : m;
            }
            stt.resc[g][tg] = ex2(old - m);
            stt.nm[g][tg] = -m;
          }
          if (tg == 0) {
            float m = cref;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, stt.wvs[g][w]);
            m = fmaxf(m, kMinVScale);
            stt.cref[g] = m;
            stt.cfac[g] = cref / m;
          }
          ptx::bar_sync(bar_id, 128);
          cref = stt.cref[g];
          if (has_o) {
#pragma unroll
            for (int j = 0; j < GP / 2; ++j) {
              const float2 f = *reinterpret_cast<const float2*>(&stt.resc[g][2 * j]);
              l2[j] = make_float2(l2[j].x * f.x, l2[j].y * f.y);
            }
            // the group's last output MMA is done before its sums are scaled
            ok = warp_wait_bounded(pe0 + 8u * g, (n_tile & 1u) ^ 1u, abort_flag, &g_attn_watchdog, kSiteAccEmpty) && ok;
            ptx::tc_fence_after();
            const float cf = stt.cfac[g];
#pragma unroll 1
            for (int b = 0; b < N2; b += 16) {
              uint32_t r[16];
              ptx::tmem_ld_32x32b_x16(o_tm + b, r);
              ptx::tmem_wait_ld_n(r);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) * (stt.resc[g][(b + j) % GP] * cf));
              ptx::tmem_st_32x32b_x16(o_tm + b, r);
            }
            ptx::tmem_wait_st();
          }
        }
        if (!any) continue;
        // ---- probabilities; P is free once the group's last output MMA is done
        ok = warp_wait_bounded(pe0 + 8u * g, (n_tile & 1u) ^ 1u, abort_flag, &g_attn_watchdog, kSiteAccEmpty) && ok;
        const float w = vs * (kPScale / cref);
        const float2 w2 = make_float2(w, w);
#pragma unroll
        for (int b = 0; b < GP; b += 16) {
          uint32_t hi[16], lo[16];
          ptx::tmem_ld_32x32b_x16(s_tm + b, hi);
          ptx::tmem_ld_32x32b_x16(s_tm + GP + b, lo);
          ptx::tmem_wait_ld_n(hi);
          ptx::tmem_wait_ld_n(lo);
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 nm = nm4[(b + j) / 4];
            uint32_t hc[2], lc[2];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float2 raw = __ffma2_rn(make_float2(__uint_as_float(lo[j + k]), __uint_as_float(lo[j + k + 1])), k16,
                                            make_float2(__uint_as_float(hi[j + k]), __uint_as_float(hi[j + k + 1])));
              const float2 t2 = __ffma2_rn(raw, c2, k == 0 ? make_float2(nm.x, nm.y) : make_float2(nm.z, nm.w));
              const float2 e2 = make_float2(ex2(t2.x), ex2(t2.y));
              float2& l = l2[(b + j + k) / 2];
              l = __fadd2_rn(l, e2);
              const float2 pw = __fmul2_rn(e2, w2);
              split_pair(__floats2half2_rn(pw.x, pw.y), &hc[k / 2], &lc[k / 2]);
            }
            ph[j / 4] = hc[0] | hc[1] << 16;
            pl[j / 4] = lc[0] | lc[1] << 16;
          }
          *reinterpret_cast<uint4*>(p_row + (((b / 16) ^ p_swz) << 4)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
          *reinterpret_cast<uint4*>(p_row + ((((GP + b) / 16) ^ p_swz) << 4)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(se0 + 8u * g);
          ptx::mbar_arrive(pf0 + 8u * g);
        }
        has_o = true;
        ++n_tile;
      }
      if (stop) break;

      // ---- the unit's end: both groups' sums and maxima meet
      if (has_o) {
        warp_wait_bounded(pe0 + 8u * g, (n_tile & 1u) ^ 1u, abort_flag, &g_attn_watchdog, kSiteAccEmpty);
      }
#pragma unroll
      for (int j = 0; j < GP / 2; ++j) {
        float2 v = l2[j];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          v.x += __shfl_xor_sync(kFull, v.x, d);
          v.y += __shfl_xor_sync(kFull, v.y, d);
        }
        if (lane == 0) *reinterpret_cast<float2*>(&stt.lred[par][g][quad][2 * j]) = v;
      }
      if (tg < GP) stt.msave[par][g][tg] = has_o ? -stt.nm[g][tg] : kMinM;
      if (tg == 0) {
        stt.csave[par][g] = cref;
        stt.used[par][g] = has_o ? 1.f : 0.f;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ub);
      warp_wait_bounded(ub, i & 1, abort_flag, &g_attn_watchdog, kSiteAccFull);
      ptx::tc_fence_after();
      int row, kvh, h0;
      unit_of(p, u0 + i * ustep, &row, &kvh, &h0, GP);
      const int nh = min(GP, p.group - h0);
      constexpr int kHalf = GP / 2;  // group g finishes heads [g*kHalf, (g+1)*kHalf)
      if (tg < kHalf) {
        const int h = g * kHalf + tg;
        float ls[2], ms[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ms[k] = stt.msave[par][k][h];
          ls[k] = (stt.lred[par][k][0][h] + stt.lred[par][k][1][h]) + (stt.lred[par][k][2][h] + stt.lred[par][k][3][h]);
        }
        const float m = (ms[0] > ms[1] || ms[0] != ms[0]) ? ms[0] : ms[1];
        float f[2], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f[k] = stt.used[par][k] != 0.f ? ex2(ms[k] - m) : 0.f;
          sum += f[k] * ls[k];
        }
        const float norm = CLUSTER ? 1.f / kPScale : sum == 0.f ? 0.f : 1.f / (sum * kPScale);
#pragma unroll
        for (int k = 0; k < 2; ++k) stt.fac[h][k] = f[k] * stt.csave[par][k] * norm;
        if constexpr (CLUSTER) {
          stt.xm[h] = m;
          stt.xl[h] = sum;
        } else if (p.lse != nullptr && h < nh) {
          p.lse[static_cast<int64_t>(row) * p.heads + kvh * p.group + h0 + h] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
        }
      }
      const bool used0 = stt.used[par][0] != 0.f, used1 = stt.used[par][1] != 0.f;
      ptx::bar_sync(bar_id, 128);
      const int ch = D == 128 ? tg : tg - 64;  // D = 64: the value half of the shared rows
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row / p.next_n * p.out_req_stride +
                           row % p.next_n * p.out_row_stride + (kvh * p.group + h0) * p.out_head_stride + ch;
      float* xo = reinterpret_cast<float*>(smem + L.kv);  // cluster: [GP][128], where the tiles were
#pragma unroll 1
      for (int b = g * kHalf; b < (g + 1) * kHalf; b += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k == 0 ? used0 : used1) {
            const uint32_t o = tmem + (2 + k) * N2 + lane_off + b;
            uint32_t hi[8], lo[8];
            ptx::tmem_ld_32x32b_x8(o, hi);
            ptx::tmem_ld_32x32b_x8(o + GP, lo);
            ptx::tmem_wait_ld_n(hi);
            ptx::tmem_wait_ld_n(lo);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = fmaf(fmaf(__uint_as_float(lo[j]), 0.0625f, __uint_as_float(hi[j])), stt.fac[b + j][k], v[j]);
          }
        }
        if constexpr (CLUSTER) {
#pragma unroll
          for (int j = 0; j < 8; ++j) xo[(b + j) * 128 + tg] = v[j];
        } else if (ch >= 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (b + j < nh) out[(b + j) * p.out_head_stride] = __float2bfloat16(v[j]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(oe);
    }
  }

  if constexpr (CLUSTER) {
    // ---- the CTAs' shares meet: CTA r finishes heads [r*GP/C, (r+1)*GP/C)
    cg::cluster_group cl = cg::this_cluster();
    __syncwarp();
    cl.sync();
    if (warp < 4 * kAttnGroups && n_units > 0) {
      const int tg = threadIdx.x & 127, half = threadIdx.x >> 7;
      const int ch = D == 128 ? tg : tg - 64;
      int row, kvh, h0;
      unit_of(p, u0, &row, &kvh, &h0, GP);
      const int nh = min(GP, p.group - h0);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row / p.next_n * p.out_req_stride +
                           row % p.next_n * p.out_row_stride + (kvh * p.group + h0) * p.out_head_stride + ch;
      const int h_end = min(nh, (crank + 1) * GP / C);
      for (int h = crank * GP / C + half; h < h_end; h += 2) {
        float m = kMinM;
        for (int r = 0; r < C; ++r) {
          const float x = *cl.map_shared_rank(&stt.xm[h], r);
          m = (x > m || x != x) ? x : m;
        }
        float sum = 0.f, v = 0.f;
        for (int r = 0; r < C; ++r) {
          const float f = ex2(*cl.map_shared_rank(&stt.xm[h], r) - m);
          sum = fmaf(f, *cl.map_shared_rank(&stt.xl[h], r), sum);
          v = fmaf(f, *cl.map_shared_rank(reinterpret_cast<float*>(smem + L.kv) + h * 128 + tg, r), v);
        }
        if (ch >= 0) out[h * p.out_head_stride] = __float2bfloat16(sum == 0.f ? 0.f : v / sum);
        if (p.lse != nullptr && tg == 0)
          p.lse[static_cast<int64_t>(row) * p.heads + kvh * p.group + h0 + h] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      }
    }
    __syncwarp();
    cl.sync();  // no CTA leaves while another reads its shared memory
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

namespace {
using AttnKernel = void (*)(CUtensorMap, SparseAttnParams);
template <int D, bool CLUSTER>
AttnKernel attn_instance(int gp) {
  return gp == 16   ? sparse_attn_kernel<D, 16, CLUSTER>
         : gp == 32 ? sparse_attn_kernel<D, 32, CLUSTER>
                    : sparse_attn_kernel<D, 64, CLUSTER>;
}
}  // namespace

cudaError_t launch_sparse_attn(const CUtensorMap& tm_kv, const SparseAttnParams& p, int head_dim, int grid, int ctas,
                               int smem_bytes, cudaStream_t stream) {
  const int gp = attn_pad(p.group);
  const AttnKernel kern = head_dim == 128 ? (ctas > 1 ? attn_instance<128, true>(gp) : attn_instance<128, false>(gp))
                                          : (ctas > 1 ? attn_instance<64, true>(gp) : attn_instance<64, false>(gp));
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem_bytes);
  if (e != cudaSuccess) return e;
  if (ctas == 1) {
    kern<<<grid, kAttnThreads, smem_bytes, stream>>>(tm_kv, p);
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
  return cudaLaunchKernelEx(&cfg, kern, tm_kv, p);
}

cudaError_t read_attn_watchdog(unsigned int* value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_attn_watchdog, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_attn_watchdog, &zero, sizeof(unsigned int));
}

}  // namespace fp8idx
