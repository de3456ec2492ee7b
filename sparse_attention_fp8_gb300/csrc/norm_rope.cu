// Norms of the heads' queries and keys and the rotation of their positions in
// one pass (fp8idx_head_norm_rope).
//
// A row is one head of one token.  D/8 lanes hold it, eight values each: sums
// are butterflies among them, and the value that a rotation pairs with another
// one is in the same lane (neighbouring pairs) or in the lane rot/16 further on
// (halves), which takes one exchange.  A warp keeps to one token and walks its
// heads, so the token's sines and cosines are made once, in the registers of
// the lanes that need them, and no table of them is read.
//
// Angles of far positions: position * inv_freq has up to 55 bits, of which the
// whole turns do not matter.  inv_freq / 2 pi becomes a 64-bit fraction of a
// turn (a product of the float's significand with 1/(2 pi) in whole numbers),
// its product with the position wraps at whole turns by itself, and the upper
// 32 bits are the angle to 2^-32 turns, exactly reduced to an eighth of a turn
// around zero, where the Taylor series of sine and cosine to x^9 and x^10 are
// good to 2e-9; with the f32 roundings of the angle and the series a cosine is off
// by 1.02e-7 at most and a sine by 9.1e-8 (over all 2^30 reduced angles), and by
// 1.5e-9 for the angle's last bit.  (In 32-bit floats the product alone would be
// off by 0.004 at position 100000; 64-bit floats run at a sixty-fourth of the rate
// here.)
// DRAM bound: every value is read and written once.  16384 tokens of 32 + 8 bf16
// heads of 128 take 55.3 us, 6.07 TB/s of the 6.68 that a copy reaches, f32 heads
// 100.5 us, 6.68 TB/s; one token 3.3 us, a launch.
#include <cuda_runtime.h>

#include <type_traits>

#include "rows.cuh"

namespace fp8idx {
namespace {

constexpr int kNormRopeThreads = 128;
constexpr uint32_t kFull = 0xffffffffu;

// f / (2 pi) turns as a fraction of 2^64, whole turns dropped.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  // 1 / (2 pi) * 2^66 (its first two bits are zeros), and 64 more bits
  constexpr uint64_t kHi = 0xA2F9836E4E441529ull, kLo = 0xFC2757D1F534DDC0ull;
  const uint32_t bits = __float_as_uint(f), field = bits >> 23 & 0xFFu;
  const uint64_t m = (bits & 0x7FFFFFu) | (field ? 0x800000u : 0u);
  // m * 1/(2 pi) * 2^66, below 2^88, times 2^(exponent - 2)
  const uint64_t carry = __umul64hi(m, kLo), low = m * kHi + carry;
  const uint64_t high = __umul64hi(m, kHi) + (low < carry ? 1u : 0u);
  const int right = 152 - static_cast<int>(field ? field : 1u);  // 2 - (field - 150)
  uint64_t t;
  if (right >= 128)
    t = 0;
  else if (right >= 64)
    t = high >> (right - 64);
  else if (right > 0)
    t = high << (64 - right) | low >> right;
  else
    t = right > -64 ? low << -right : 0;
  return bits >> 31 ? 0 - t : t;
}

// cosine and sine of `position` times `turn` 2^-64 turns, times `mul`.
__device__ __forceinline__ void rotation(int32_t position, float inv_freq, float mul, float* c, float* s) {
  const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(position)) * turn_fraction(inv_freq);
  const uint32_t phase = static_cast<uint32_t>((at + 0x80000000ull) >> 32);
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(phase - (quarter << 30))) * 1.46291807926716e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float sn = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  sn = fmaf(x2, sn, 8.33333333e-3f);
  sn = fmaf(x2, sn, -1.66666667e-1f);
  sn = fmaf(x2 * x, sn, x);
  float cs = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
  cs = fmaf(x2, cs, -1.38888889e-3f);
  cs = fmaf(x2, cs, 4.16666667e-2f);
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.f);
  const float a = quarter & 1u ? sn : cs, b = quarter & 1u ? cs : sn;
  *c = ((quarter + 1u) & 2u ? -a : a) * mul;
  *s = (quarter & 2u ? -b : b) * mul;
}

template <int TYPE>
__device__ __forceinline__ void store8(uint8_t* dst, const float (&y)[8]) {
  uint4* d = reinterpret_cast<uint4*>(dst);
  if constexpr (TYPE == kRowF32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __stcs(d + i, make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                               __float_as_uint(y[4 * i + 3])));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kRowBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    __stcs(d, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

}  // namespace

// L lanes a row (8, 16 or 32; those past D/8 idle); PAIRS: neighbouring pairs
// are rotated, else halves of the rotated part.
template <int TYPE, int L, bool PAIRS>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_kernel(const NormRopeParams p) {
  // Rows that a warp holds side by side, and of those in flight (4099 tokens of
  // 24 f32 heads of 64: 15.8 us with 2, 13.9 with 3, 14.8 with 4, 18.0 with 8).
  constexpr int kRows = 32 / L, kBatch = 3;
  constexpr int kItem = TYPE == kRowF32 ? 4 : 2;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const uint32_t warp = blockIdx.x * (kNormRopeThreads / 32) + (threadIdx.x >> 5);
  const uint32_t t = warp / static_cast<uint32_t>(p.chunks);
  if (t >= static_cast<uint32_t>(p.tokens)) return;
  const int32_t position = __ldg(p.positions + t);
  if (position < 0) return;
  const bool live = sub < p.dim / 8;
  // The warp's groups of rows (queries', then keys').
  const int chunk = static_cast<int>(warp - t * p.chunks), from = chunk * p.per, to = min(from + p.per, p.groups[0] + p.groups[1]);
  Raw8<TYPE> raw[kBatch] = {};
  const auto load = [&](int side, int at, int end) {
    const uint8_t* const x = static_cast<const uint8_t*>(p.x[side]) + t * p.x_token[side] + sub * 8 * kItem;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = (at + i) * kRows + lane / L;
      if (live && at + i < end && h < p.heads[side]) raw[i].load(x + h * p.x_head[side]);
    }
  };
  const int first_side = from >= p.groups[0] ? 1 : 0;
  load(first_side, first_side ? from - p.groups[0] : from, first_side ? to - p.groups[0] : min(to, p.groups[0]));

  // The rotation of this lane's values: its first value's place in the rotated part.
  const int rel = sub * 8 - p.rot_start, half = p.rot / 2;
  const bool turns = live && rel >= 0 && rel < p.rot;
  constexpr int kAngles = PAIRS ? 4 : 8;
  float cs[kAngles], sn[kAngles];
  int partner = lane;
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rotation(position, turns ? __ldg(p.inv_freq + rel / 2 + i) : 0.f, p.rope_scale, &cs[i], &sn[i]);
  } else {
    // a lane and its partner have the same eight angles: each makes four
    const bool upper = turns && rel >= half;
    if (turns) partner = lane + (upper ? -half : half) / 8;
    float c4[4], s4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rotation(position, turns ? __ldg(p.inv_freq + (upper ? rel - half + 4 : rel) + i) : 0.f, p.rope_scale, &c4[i], &s4[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = __shfl_sync(kFull, c4[i], partner), s = __shfl_sync(kFull, s4[i], partner);
      cs[i] = upper ? c : c4[i];
      cs[i + 4] = upper ? c4[i] : c;
      sn[i] = upper ? s : -s4[i];
      sn[i + 4] = upper ? s4[i] : -s;
    }
  }
#pragma unroll 1
  for (int side = first_side; side < 2; ++side) {
    const int base = side ? p.groups[0] : 0, end = min(to - base, p.groups[side]), begin = max(from - base, 0);
    if (begin >= end) continue;
    float w[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = live && p.weight[side] ? __ldg(p.weight[side] + sub * 8 + i) : 1.f;
      b[i] = live && p.bias[side] ? __ldg(p.bias[side] + sub * 8 + i) : 0.f;
    }
    uint8_t* const y = static_cast<uint8_t*>(p.y[side]) + t * p.y_token[side] + sub * 8 * kItem;
#pragma unroll 1
    for (int at = begin; at < end; at += kBatch) {
      if (at > begin || side != first_side) load(side, at, end);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (at + i >= end) break;  // (the same for the whole warp)
        const int h = (at + i) * kRows + lane / L;
        float v[8];
        raw[i].values(v);
        if (p.norm == kNormLayer) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += v[j];
          const float mean = row_sum<L>(sum) * p.inv_dim;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = live ? v[j] - mean : 0.f;
        }
        if (p.norm != kNormNone) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
          const float r = rsqrtf(fmaf(row_sum<L>(sum), p.inv_dim, p.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j] * r, w[j], b[j]);
        }
        float out[8];
        if constexpr (PAIRS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = v[2 * j], c = v[2 * j + 1];
            out[2 * j] = turns ? fmaf(a, cs[j], -(c * sn[j])) : a;
            out[2 * j + 1] = turns ? fmaf(c, cs[j], a * sn[j]) : c;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float other = __shfl_sync(kFull, v[j], partner);
            out[j] = turns ? fmaf(v[j], cs[j], other * sn[j]) : v[j];
          }
        }
        if (live && h < p.heads[side]) store8<TYPE>(y + h * p.y_head[side], out);
      }
    }
  }
}

namespace {
// Four values as they lie in memory.
template <int TYPE>
struct Raw4 {
  using Word = typename std::conditional<TYPE == kRowF32, uint4, uint2>::type;
  Word v;
  __device__ __forceinline__ void load(const uint8_t* src) { v = __ldcs(reinterpret_cast<const Word*>(src)); }
  __device__ __forceinline__ void values(float2 (&x)[2]) const {
    if constexpr (TYPE == kRowF32) {
      x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
      x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    } else if constexpr (TYPE == kRowBf16) {
      x[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
      x[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
    } else {
      x[0] = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
      x[1] = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[2]) {
    if constexpr (TYPE == kRowF32) {
      v = make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    } else if constexpr (TYPE == kRowBf16) {
      const __nv_bfloat162 a = __float22bfloat162_rn(x[0]), b = __float22bfloat162_rn(x[1]);
      v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __half2 a = __float22half2_rn(x[0]), b = __float22half2_rn(x[1]);
      v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
};
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }
}  // namespace

// Halves of the whole head, 8 * L elements: a lane has four values of each half,
// so pairs meet in it, and arithmetic goes two values an instruction (16384
// tokens of 40 heads: 55 us, where the kernel above takes 110).
template <int TYPE, int L>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_whole_kernel(const NormRopeParams p) {
  constexpr int kRows = 32 / L, kBatch = 4;  // (2: 62.9 us, 8: 58.7)
  constexpr int kPiece = TYPE == kRowF32 ? 16 : 8, kHalf = L * kPiece;  // bytes of four values, of half a row
  const int lane = threadIdx.x & 31, sub = lane % L;
  const uint32_t warp = blockIdx.x * (kNormRopeThreads / 32) + (threadIdx.x >> 5);
  const uint32_t t = warp / static_cast<uint32_t>(p.chunks);
  if (t >= static_cast<uint32_t>(p.tokens)) return;
  const int32_t position = __ldg(p.positions + t);
  if (position < 0) return;
  const int chunk = static_cast<int>(warp - t * p.chunks), from = chunk * p.per, to = min(from + p.per, p.groups[0] + p.groups[1]);
  float2 cs[2], sn[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    rotation(position, __ldg(p.inv_freq + sub * 4 + 2 * i), p.rope_scale, &cs[i].x, &sn[i].x);
    rotation(position, __ldg(p.inv_freq + sub * 4 + 2 * i + 1), p.rope_scale, &cs[i].y, &sn[i].y);
  }
#pragma unroll 1
  for (int side = from >= p.groups[0] ? 1 : 0; side < 2; ++side) {
    const int base = side ? p.groups[0] : 0, end = min(to - base, p.groups[side]), begin = max(from - base, 0);
    if (begin >= end) continue;
    float2 w[2][2], b[2][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (i / 4) * 4 * L + sub * 4 + i % 4;
      const float wi = p.weight[side] ? __ldg(p.weight[side] + e) : 1.f, bi = p.bias[side] ? __ldg(p.bias[side] + e) : 0.f;
      float2 &w2 = w[i / 4][i % 4 / 2], &b2 = b[i / 4][i % 4 / 2];
      (i % 2 ? w2.y : w2.x) = wi;
      (i % 2 ? b2.y : b2.x) = bi;
    }
    const int heads = p.heads[side];
    const uint8_t* x = static_cast<const uint8_t*>(p.x[side]) + t * p.x_token[side] + sub * kPiece;
    uint8_t* y = static_cast<uint8_t*>(p.y[side]) + t * p.y_token[side] + sub * kPiece;
    int h = begin * kRows + lane / L;
    x += h * p.x_head[side];
    y += h * p.y_head[side];
    const int64_t x_step = kRows * p.x_head[side], y_step = kRows * p.y_head[side];
#pragma unroll 1
    for (int at = begin; at < end; at += kBatch) {
      Raw4<TYPE> raw[kBatch][2] = {};
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (at + i < end && h + i * kRows < heads) {
          raw[i][0].load(x + i * x_step);
          raw[i][1].load(x + i * x_step + kHalf);
        }
      x += kBatch * x_step;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (at + i >= end) break;  // (the same for the whole warp)
        float2 v[2][2];
        raw[i][0].values(v[0]);
        raw[i][1].values(v[1]);
        if (p.norm == kNormLayer) {
          const float2 sum = __fadd2_rn(__fadd2_rn(v[0][0], v[0][1]), __fadd2_rn(v[1][0], v[1][1]));
          const float2 mean = twice(-row_sum<L>(sum.x + sum.y) * p.inv_dim);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j / 2][j % 2] = __fadd2_rn(v[j / 2][j % 2], mean);
        }
        if (p.norm != kNormNone) {
          float2 sum = __fmul2_rn(v[0][0], v[0][0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) sum = __ffma2_rn(v[j / 2][j % 2], v[j / 2][j % 2], sum);
          const float2 r = twice(rsqrtf(fmaf(row_sum<L>(sum.x + sum.y), p.inv_dim, p.eps)));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j / 2][j % 2] = __ffma2_rn(__fmul2_rn(v[j / 2][j % 2], r), w[j / 2][j % 2], b[j / 2][j % 2]);
        }
        float2 out[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          out[0][j] = __ffma2_rn(v[0][j], cs[j], minus(__fmul2_rn(v[1][j], sn[j])));
          out[1][j] = __ffma2_rn(v[1][j], cs[j], __fmul2_rn(v[0][j], sn[j]));
        }
        if (h < heads) {
          Raw4<TYPE> o;
          o.set(out[0]);
          __stcs(reinterpret_cast<typename Raw4<TYPE>::Word*>(y), o.v);
          o.set(out[1]);
          __stcs(reinterpret_cast<typename Raw4<TYPE>::Word*>(y + kHalf), o.v);
        }
        h += kRows;
        y += y_step;
      }
    }
  }
}

namespace {
using NormRopeKernel = void (*)(NormRopeParams);
template <int TYPE, int L>
NormRopeKernel norm_rope_instance(bool pairs) {
  return pairs ? norm_rope_kernel<TYPE, L, true> : norm_rope_kernel<TYPE, L, false>;
}
template <int TYPE>
NormRopeKernel norm_rope_instance(int lanes, bool pairs, bool whole) {
  if (whole && !pairs)
    return lanes == 8 ? norm_rope_whole_kernel<TYPE, 8> : lanes == 16 ? norm_rope_whole_kernel<TYPE, 16> : norm_rope_whole_kernel<TYPE, 32>;
  return lanes == 8 ? norm_rope_instance<TYPE, 8>(pairs)
         : lanes == 16 ? norm_rope_instance<TYPE, 16>(pairs) : norm_rope_instance<TYPE, 32>(pairs);
}
}  // namespace

cudaError_t launch_norm_rope(NormRopeParams& p, int row_type, bool pairs, int sms, cudaStream_t stream) {
  const int lanes = p.dim <= 64 ? 8 : p.dim <= 128 ? 16 : 32, rows = 32 / lanes;
  for (int i = 0; i < 2; ++i) p.groups[i] = (p.heads[i] + rows - 1) / rows;
  // Groups that a warp walks: a whole token's once that leaves every SM 24 warps
  // (4099 tokens of 7 groups: 13.9 us; pieces of a token, at 32 or 64 warps,
  // 16.6 and 18.6: each makes the token's angles again), fewer below (96 tokens
  // of 20 groups: 3.7 us, with a warp for a token 6.8).
  const int groups = p.groups[0] + p.groups[1];
  const int64_t per = static_cast<int64_t>(p.tokens) * groups / (24 * sms);
  p.per = static_cast<int32_t>(per < 1 ? 1 : per > groups ? groups : per);
  p.chunks = (groups + p.per - 1) / p.per;
  const int64_t warps = static_cast<int64_t>(p.tokens) * p.chunks;
  const bool whole = p.rot == p.dim && p.dim == 8 * lanes;
  const NormRopeKernel kern = row_type == kRowBf16  ? norm_rope_instance<kRowBf16>(lanes, pairs, whole)
                              : row_type == kRowF16 ? norm_rope_instance<kRowF16>(lanes, pairs, whole)
                                                    : norm_rope_instance<kRowF32>(lanes, pairs, whole);
  constexpr int kWarps = kNormRopeThreads / 32;
  kern<<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kNormRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp8idx
