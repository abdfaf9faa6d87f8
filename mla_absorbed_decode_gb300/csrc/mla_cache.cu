// The latent cache over a request's life: RoPE with several position axes, the write of
// new rows into the paged cache (bf16, E4M3 or 4 bits), and eviction by accumulated attention
// weight.  C entries at the end (declared in mla.h).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "mla_fp4.cuh"
#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr int kRopeMaxAxes = 4;
constexpr int kPairs = 32;              // rotated pairs of a 64-value row
constexpr int kMaxRows = 1 << 30;       // rows of a call (row numbers are ints)

// Inverse frequencies theta^(-2j/64) and 2*pi as float pairs (hi + lo), and each pair's axis.
struct RopeTable {
  float hi[kPairs], lo[kPairs];
  float two_pi_hi, two_pi_lo;
  uint8_t axis[kPairs];
};

// cos and sin of an angle pos * (hi + lo): the arithmetic of rope_row (mla_rope.cuh), whose
// argument reduction keeps the angle within ~1e-7 rad for |pos| < 2^24.
__device__ __forceinline__ float2 rope_turn(const RopeTable& t, float hi, float lo, int pos) {
  const float fp = static_cast<float>(pos);
  const float inv_two_pi = 1.0f / t.two_pi_hi;
  const float a_hi = fp * hi;
  const float a_lo = fmaf(fp, lo, fmaf(fp, hi, -a_hi));
  const float k = rintf(a_hi * inv_two_pi);
  const float r = fmaf(-k, t.two_pi_lo, fmaf(-k, t.two_pi_hi, a_hi)) + a_lo;
  float sn, cs;
  __sincosf(r, &sn, &cs);   // |r| <= pi + 1e-6: the hardware sine/cosine, absolute error < 2^-21
  return make_float2(cs, sn);
}

// A value as the sum of two floats.
struct Float2Sum {
  float hi, lo;
};
__device__ __forceinline__ Float2Sum add_exactly(Float2Sum a, Float2Sum b) {   // (up to the sum of the low parts)
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  return {s, __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)) + (a.lo + b.lo)};
}
__device__ __forceinline__ Float2Sum times(float a, Float2Sum b) {
  const float p = __fmul_rn(a, b.hi);
  return {p, fmaf(a, b.hi, -p) + a * b.lo};
}
// v / d, d > 0, to 24 bits with the last bit set where bits are lost (toward zero): a later rounding to fewer bits then falls as that
// of the quotient itself would.
__device__ __forceinline__ float quotient_for_rounding(Float2Sum v, Float2Sum d) {
  const float q = __fdiv_rn(v.hi, d.hi), rest = fmaf(-q, d.hi, v.hi) + fmaf(-q, d.lo, v.lo);
  if (!(rest != 0.f) || q == 0.f || !(fabsf(q) <= 3.4e38f)) return q;
  return __uint_as_float((__float_as_uint(q) - ((rest < 0.f) == (q > 0.f) ? 1u : 0u)) | 1u);
}
// x0 a + x1 b, the factors sums of two floats.  One that is infinite (or passes float32's range) stays so: its low part, a difference
// of infinities, is NaN.
__device__ __forceinline__ Float2Sum dot2(float x0, Float2Sum a, float x1, Float2Sum b) {
  const Float2Sum s = add_exactly(times(x0, a), times(x1, b));
  if (!(fabsf(s.hi) <= FLT_MAX)) return {s.hi, 0.f};
  const float hi = __fadd_rn(s.hi, s.lo);
  return {hi, __fsub_rn(s.lo, __fsub_rn(hi, s.hi))};
}
// The pair (x0, x1) turned by the angle pos * (hi + lo), for codes: a value is off by 2^-25.5 of the pair's norm at most (positions
// below 2^17; 2^-21.8 up to 2^24, where half an ulp of the angle is 2^-1 and its low part carries 2^-25), where rope_turn's hardware
// sine, off by 2^-21, would move many times as many codes that lie halfway.  The angle less k quarter turns (pi / 2 in three floats,
// products with their rounding errors) is a pair of floats in [-pi / 4, pi / 4] or a little more, its sine and cosine are Taylor
// polynomials whose leading terms are added up exactly.
__device__ __forceinline__ void rope_turned(float hi, float lo, int pos, float x0, float x1, Float2Sum (&y)[2]) {
  constexpr float kQuarter1 = 0x1.921fb6p+0f, kQuarter2 = -0x1.777a5cp-25f, kQuarter3 = -0x1.ee59dap-50f;
  const float fp = static_cast<float>(pos);
  const float a = __fmul_rn(fp, hi), b = fmaf(fp, lo, fmaf(fp, hi, -a));
  float k = rintf(__fmul_rn(a, 0.636619772f));
  const float p1 = __fmul_rn(k, kQuarter1), p2 = __fmul_rn(k, kQuarter2);
  const float t = __fsub_rn(a, p1), u = __fsub_rn(t, p2), v = __fsub_rn(u, t);
  const float e = __fadd_rn(__fsub_rn(t, __fsub_rn(u, v)), __fsub_rn(-p2, v));   // (t - p2) - u
  const float l = e + ((b - fmaf(k, kQuarter1, -p1)) - fmaf(k, kQuarter3, fmaf(k, kQuarter2, -p2)));
  float r = __fadd_rn(u, l), rl = __fsub_rn(l, __fsub_rn(r, u));
  if (fabsf(r) > 1.f) {   // past 2^21 k comes out short by up to 1.1 quarter turns, too far for the polynomials (2^-18.4 at an angle of 2.4)
    const float more = rintf(__fmul_rn(r, 0.636619772f)), w = fmaf(-more, kQuarter1, r), rest = fmaf(-more, kQuarter2, rl);
    k += more;
    r = __fadd_rn(w, rest);
    rl = __fsub_rn(rest, __fsub_rn(r, w));
  }
  const float z = __fmul_rn(r, r), zl = fmaf(r, r, -z) + 2.f * r * rl;
  const float s1 = r * z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 6227020800.f, -1.f / 39916800.f), 1.f / 362880.f), -1.f / 5040.f),
                                        1.f / 120.f), -1.f / 6.f);
  const float sh = __fadd_rn(r, s1), sl = __fadd_rn(__fsub_rn(r, sh), s1) + fmaf(-0.5f * z, rl, rl);
  const float h = 0.5f * z, c0 = __fsub_rn(1.f, h);
  const float c1 = fmaf(z * z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 479001600.f, -1.f / 3628800.f), 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f),
                        -0.5f * zl);
  const float ch = __fadd_rn(c0, c1);
  const float cl = __fadd_rn(__fsub_rn(c0, ch), c1) + __fsub_rn(__fsub_rn(1.f, c0), h);
  const int quarter = static_cast<int>(k);
  const bool odd = quarter & 1;
  Float2Sum sn = odd ? Float2Sum{ch, cl} : Float2Sum{sh, sl}, cs = odd ? Float2Sum{sh, sl} : Float2Sum{ch, cl};
  if (quarter & 2) sn = {-sn.hi, -sn.lo};
  if ((quarter + 1) & 2) cs = {-cs.hi, -cs.lo};
  y[0] = dot2(x0, cs, -x1, sn);
  y[1] = dot2(x0, sn, x1, cs);
}

// ------------------------------------------------------------------- rope --
struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t x_row, x_head, out_row, out_head;
  const int32_t* positions;
  int64_t pos_stride;
  int N, H;
  int log_heads;            // log2 of a token's rows in a round of 32
  float sign;               // -1: the inverse rotation
  RopeTable table;
};

// A block of 256 threads: 32 rows at a time (a thread turns 4 pairs, 16 bytes, of one row), of one token's heads or,
// below 32 heads, of several tokens; kRounds rounds of heads share the token's cosines and sines, which are
// computed once, into shared memory (each thread's own: 92 us for 4096 tokens of 128 heads, arithmetic-bound).
constexpr int kRopeMaxTokens = 32;
template <int kRounds>
__global__ void __launch_bounds__(256) mla_rope_axes_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 turns[kRopeMaxTokens][kPairs];   // (cos, sin), 16-byte units of two pairs
  griddep_wait();
  griddep_launch_dependents();
  const int tokens = 32 >> p.log_heads;              // of this block
  const int u = threadIdx.x & 7, row = threadIdx.x >> 3;   // u: pairs 4 u .. 4 u + 3
  const int tok = row >> p.log_heads, n0 = blockIdx.x * tokens;
  const int n = n0 + tok;
  const int h0 = static_cast<int>(blockIdx.y) * 32 * kRounds + (row & ((1 << p.log_heads) - 1));
  uint4 v[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (n < p.N && h0 + 32 * r < p.H)
      v[r] = *reinterpret_cast<const uint4*>(p.x + n * p.x_row + (h0 + 32 * r) * p.x_head + u * 8);
  for (int i = threadIdx.x; i < tokens * kPairs; i += 256) {
    const int j = i % kPairs, at = n0 + i / kPairs;
    if (at < p.N) {
      const float2 t = rope_turn(p.table, p.table.hi[j], p.table.lo[j],
                                 __ldg(p.positions + p.table.axis[j] * p.pos_stride + at));
      turns[i / kPairs][j] = make_float2(t.x, t.y * p.sign);
    }
  }
  __syncthreads();
  if (n >= p.N) return;
  float2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = turns[tok][4 * u + i];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (h0 + 32 * r >= p.H) break;
    uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = bf16_lo(w[i]), x1 = bf16_hi(w[i]);
      w[i] = pack_bf16x2(fmaf(x0, t[i].x, -x1 * t[i].y), fmaf(x0, t[i].y, x1 * t[i].x));
    }
    *reinterpret_cast<uint4*>(p.out + n * p.out_row + (h0 + 32 * r) * p.out_head + u * 8) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ----------------------------------------------------------------- append --
struct AppendParams {
  const __nv_bfloat16* c;
  const __nv_bfloat16* pe;
  int64_t c_row, pe_row;
  void* kv;
  int64_t num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seqlens;
  const int32_t* offsets;   // [B + 1], or nullptr: rows_each rows a request
  int N, B, rows_each;
  const int32_t* positions; // nullptr: k_pe is copied
  int64_t pos_stride;
  float kv_scale, kv_inv;
  int* status;
  const __nv_bfloat16* norm;   // 4-bit cache: [512] weights of the latent's norm, or nullptr
  float norm_eps;
  RopeTable table;
};

// The request of row r: the last b with offsets[b] <= r (-1 or B for a row of none).  The warp
// narrows [lo, hi) by 32 pivots a step, so that a batch of 16384 takes three dependent loads.
__device__ __forceinline__ int request_of(const int32_t* offsets, int B, int r, int lane) {
  int lo = 0, hi = B + 1;   // offsets[lo - 1] <= r < offsets[hi], with offsets[-1] = -inf, offsets[B + 1] = inf
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step + step - 1;
    const bool le = at < hi && __ldg(offsets + at) <= r;
    const int k = __popc(__ballot_sync(0xffffffffu, le));   // the first k pivots are <= r
    const int nlo = lo + k * step;
    hi = k == 32 ? hi : min(hi, nlo + step - 1);
    lo = min(nlo, hi);
  }
  return lo - 1;
}

// The cached row (page and slot) that new row r goes to: of request b, whose rows end before row `end`.  -1: it belongs to
// no request, or its token or page is out of range (reported).  All lanes of the warp agree.
__device__ __forceinline__ int64_t append_target(const AppendParams& p, int r, int lane) {
  int b, end;
  if (p.offsets != nullptr) {
    b = request_of(p.offsets, p.B, r, lane);
    if (b < 0 || b >= p.B) return -1;
    end = __ldg(p.offsets + b + 1);
  } else {
    b = r / p.rows_each;
    end = (b + 1) * p.rows_each;
  }
  const int64_t t = static_cast<int64_t>(__ldg(p.seqlens + b)) - (end - r);
  if (t >= 0 && t < static_cast<int64_t>(p.max_blocks) * kPageTokens) {
    const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + t / kPageTokens);
    if (blk >= 0 && blk < p.num_blocks) return static_cast<int64_t>(blk) * kPageTokens + t % kPageTokens;
  }
  if (lane == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
  return -1;
}

// One warp per new row: 64 units of 8 latent values, lane l takes units l and l + 32, and 32 pairs of k_pe, a pair a
// lane.  kDivide: an FP8 scale that is no power of two, so that x / kv_scale has to be a division (the product
// with the reciprocal is the same number for a power of two).
template <bool F8, bool kDivide>
__global__ void __launch_bounds__(128) mla_append_kernel(const __grid_constant__ AppendParams p) {
  // the table, read by the lanes at 32 different places, costs a constant-memory access 32 turns: once a block, and
  // before the wait (3.8 us for 6900 rows, 8.0 where every warp does it)
  __shared__ float s_hi[kPairs], s_lo[kPairs];
  __shared__ int s_axis[kPairs];
  const int lane = threadIdx.x & 31;
  if (p.positions != nullptr && threadIdx.x < kPairs) {
    s_hi[lane] = p.table.hi[lane];
    s_lo[lane] = p.table.lo[lane];
    s_axis[lane] = p.table.axis[lane];
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= p.N) return;
  const uint4* c = reinterpret_cast<const uint4*>(p.c + r * p.c_row);
  const uint4 c0 = __ldg(c + lane), c1 = __ldg(c + 32 + lane);
  const uint32_t pe = __ldg(reinterpret_cast<const uint32_t*>(p.pe + r * p.pe_row) + lane);
  int pos = 0;
  if (p.positions != nullptr) pos = __ldg(p.positions + s_axis[lane] * p.pos_stride + r);
  const int64_t row = append_target(p, r, lane);
  if (row < 0) return;
  float x0 = bf16_lo(pe), x1 = bf16_hi(pe);
  if (p.positions != nullptr) {
    const float2 turn = rope_turn(p.table, s_hi[lane], s_lo[lane], pos);
    const float y0 = fmaf(x0, turn.x, -x1 * turn.y), y1 = fmaf(x0, turn.y, x1 * turn.x);
    x0 = y0, x1 = y1;
  }
  if constexpr (F8) {
    uint8_t* dst = static_cast<uint8_t*>(p.kv) + row * kDimQK;
    auto code2 = [&](float a, float b2) {
      return kDivide ? cvt_e4m3x2(__fdiv_rn(a, p.kv_scale), __fdiv_rn(b2, p.kv_scale))
                     : cvt_e4m3x2(a * p.kv_inv, b2 * p.kv_inv);
    };
    auto store = [&](int u, const uint4& v) {
      *reinterpret_cast<uint2*>(dst + u * 8) =
          make_uint2(code2(bf16_lo(v.x), bf16_hi(v.x)) | (code2(bf16_lo(v.y), bf16_hi(v.y)) << 16),
                     code2(bf16_lo(v.z), bf16_hi(v.z)) | (code2(bf16_lo(v.w), bf16_hi(v.w)) << 16));
    };
    store(lane, c0);
    store(32 + lane, c1);
    *reinterpret_cast<uint16_t*>(dst + kDimV + 2 * lane) = static_cast<uint16_t>(code2(x0, x1));
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.kv) + row * kDimQK;
    reinterpret_cast<uint4*>(dst)[lane] = c0;
    reinterpret_cast<uint4*>(dst)[32 + lane] = c1;
    reinterpret_cast<uint32_t*>(dst + kDimV)[lane] = p.positions != nullptr ? pack_bf16x2(x0, x1) : pe;
  }
}

// A row of the 4-bit cache (mla_fp4.cuh) from one new row, one warp a row: a lane has one group of 16 latent values, which
// it normalises, scales and rounds, and one pair of k_pe.
//   y = c, or c * rsqrt(mean(c^2) + eps) * w;  scale = E4M3(max|y| / (6 kv_scale));  code = E2M1(y / (scale kv_scale))
// Codes that lie halfway are few but a flipped scale moves its whole group, so what is rounded is known to more than fp32's 24 bits:
// values, scales and quotients are sums of two floats, and codes come out as from 64 bits.  The codes' quotients are formed only
// where products with a little less and a little more than the factor (off by 2^-21 at most with all roundings, the margin is 2^-20)
// round to different ones.  Values of a group whose scale rounds to 0 are stored as 0.
// 32768 rows without a norm 19.5 us (replayed from a graph for milliseconds), 49 MB: the instructions bound it, 490 a row, not the
// bytes (7 us); 6890 rows with a norm 8.4 us, 780 a row.
template <bool Norm>
__global__ void __launch_bounds__(128) mla_append_fp4_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float s_hi[kPairs], s_lo[kPairs];
  __shared__ int s_axis[kPairs];
  const int lane = threadIdx.x & 31;
  if (p.positions != nullptr && threadIdx.x < kPairs) {
    s_hi[lane] = p.table.hi[lane];
    s_lo[lane] = p.table.lo[lane];
    s_axis[lane] = p.table.axis[lane];
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= p.N) return;
  const uint4* c = reinterpret_cast<const uint4*>(p.c + r * p.c_row) + 2 * lane;
  const uint4 c0 = __ldg(c), c1 = __ldg(c + 1);
  const uint32_t pe = __ldg(reinterpret_cast<const uint32_t*>(p.pe + r * p.pe_row) + lane);
  int pos = 0;
  if (p.positions != nullptr) pos = __ldg(p.positions + s_axis[lane] * p.pos_stride + r);
  uint4 w0 = {}, w1 = {};
  if constexpr (Norm) {
    w0 = __ldg(reinterpret_cast<const uint4*>(p.norm) + 2 * lane);
    w1 = __ldg(reinterpret_cast<const uint4*>(p.norm) + 2 * lane + 1);
  }
  const int64_t row = append_target(p, r, lane);
  if (row < 0) return;
  Float2Sum rope[2] = {{bf16_lo(pe), 0.f}, {bf16_hi(pe), 0.f}};
  if (p.positions != nullptr) rope_turned(s_hi[lane], s_lo[lane], pos, rope[0].hi, rope[1].hi, rope);
  const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  float y[16];                     // the values are y * inv
  Float2Sum inv = {1.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) y[2 * i] = bf16_lo(cw[i]), y[2 * i + 1] = bf16_hi(cw[i]);
  if constexpr (Norm) {
    Float2Sum ss;
    auto mean_square = [&](float eps) {   // of the warp's row, and eps (squares of bf16 are exact where they are normal)
      ss = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = add_exactly(ss, {__fmul_rn(y[i], y[i]), 0.f});
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss = add_exactly(ss, {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
      ss = add_exactly({ss.hi * (1.f / kDimV), ss.lo * (1.f / kDimV)}, {eps, 0.f});
    };
    mean_square(p.norm_eps);
    if (!(ss.hi >= 0x1p-80f && ss.hi <= 0x1p120f)) {
      // Squares that float32 has no room for (all lanes agree): the row, and eps with it, by a power of two that brings the larger of
      // the row's largest element and sqrt(eps) to [1, 4), and the same result.  Not for rows of zeros, or with an infinity or NaN.
      uint32_t top = __float_as_uint(sqrtf(p.norm_eps));
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
      top = __reduce_max_sync(0xffffffffu, top);
      if (top > 0u && top < 0x7F800000u) {
        const float by = __uint_as_float((254u - min(top >> 23, 253u)) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] *= by;
        mean_square(p.norm_eps * by * by);
      }
    }
    // its inverse root: an approximation and one step of Newton's method for the rest, then a power of two times a number in [1, 2)
    const float r = rsqrtf(ss.hi);
    const Float2Sum rr = times(r, {r, 0.f}), one = times(ss.hi, rr);
    const float rest = 0.5f * r * (((1.f - one.hi) - one.lo) - ss.lo * rr.hi);
    const uint32_t bits = __float_as_uint(r), e = bits >> 23;
    float p2 = r;
    if (e > 0 && e < 254 && fabsf(rest) < r) {   // (not for rows of zeros or with infinities)
      p2 = __uint_as_float(e << 23);
      inv = {__uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u), rest * __uint_as_float((254u - e) << 23)};
    }
    const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) y[2 * i] = y[2 * i] * p2 * bf16_lo(ww[i]), y[2 * i + 1] = y[2 * i + 1] * p2 * bf16_hi(ww[i]);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(y[i]));
  const uint32_t scale = cvt_e4m3x2(quotient_for_rounding(times(amax, inv), times(6.f, {p.kv_scale, 0.f})), 0.f) & 0xFFu;
  const Float2Sum step = times(e4m3x2_to_float2(scale).x, {p.kv_scale, 0.f});
  uint32_t code[2] = {0u, 0u};
  if (step.hi > 0.f) {   // (no group whose scale is 0 or NaN)
    const float f = __frcp_rn(step.hi) * inv.hi, less = f * (1.f - 0x1p-20f), more = f * (1.f + 0x1p-20f);
    uint32_t other[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      code[i >> 2] |= cvt_e2m1x2(y[2 * i] * less, y[2 * i + 1] * less) << (8 * (i & 3));
      other[i >> 2] |= cvt_e2m1x2(y[2 * i] * more, y[2 * i + 1] * more) << (8 * (i & 3));
    }
    if (code[0] != other[0] || code[1] != other[1]) {
      code[0] = code[1] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        code[i >> 2] |= cvt_e2m1x2(quotient_for_rounding(times(y[2 * i], inv), step), quotient_for_rounding(times(y[2 * i + 1], inv), step))
                        << (8 * (i & 3));
    }
  }
  uint8_t* dst = static_cast<uint8_t*>(p.kv) + row * kFp4RowBytes;
  *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(code[0], code[1]);
  dst[kFp4Scales + lane] = static_cast<uint8_t>(scale);
  *reinterpret_cast<uint16_t*>(dst + kFp4Rope + 2 * lane) =
      static_cast<uint16_t>(cvt_e4m3x2(quotient_for_rounding(rope[0], {p.kv_scale, 0.f}), quotient_for_rounding(rope[1], {p.kv_scale, 0.f})));
}

// ------------------------------------------------------------------ evict --
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelDigitBits = 11, kSelBins = 1 << kSelDigitBits;   // three digits: 11, 11 and 10 bits
constexpr int kSelMaxCtas = 8;          // CTAs of a request's cluster
constexpr int kSelSlotsPerCta = 4096;   // a request gets another CTA for every so many slots
constexpr int kEvictMaxSlots = 262144;  // 32768 keys a CTA: 128 KiB of shared memory, and 16 bits a count
constexpr int kMoveSlots = 12;          // slots of one warp of the move kernel

struct EvictParams {
  void* kv;
  int64_t num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seqlens;
  const float* weights;
  int64_t weights_stride;
  const int32_t* arrival;
  int64_t arrival_stride;
  int budget, sink, recent, slots;
  int sel_log_slice;        // selection: log2 of the slots of a CTA
  int32_t* new_seqlens;
  int32_t* kept;
  float* weights_out;
  int32_t* arrival_out;
  int64_t width;
  int* status;
};

// Order of a weight as an unsigned number: larger is kept first, NaN is 0 and no weight is the
// largest number (which stands for a guarded token).
__device__ __forceinline__ uint32_t weight_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 + 0 = +0
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {   // CTA `rank`'s copy of *p
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld_cluster_v2(const uint2* p, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}
// The cluster's last barrier: what its threads have read of one another has arrived (it is in their outputs), and what
// they have written is nobody's here, so nothing is released (39.4 -> 38.9 us for 4 requests of 131072 slots).
__device__ __forceinline__ void cluster_done() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Asynchronous copy of 4 bytes global -> shared.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

struct alignas(16) SelShared {
  uint32_t hist[3][kSelBins / 2];   // bins in descending order of their digit, two 16-bit counts a word
  uint32_t warp_sum[kSelWarps];
  uint32_t digit, need, here;   // the digit in which the m-th largest key lies; keys wanted of it, keys there
  uint32_t kept, below;         // this CTA's kept slots; those of them below slot m
  int newest;                   // this CTA's largest arrival number
};
// Dynamic shared memory of a CTA with `slice` slots: keys (later the list of sources), keep mask, prefix counts.
__host__ __device__ constexpr size_t sel_smem(int slice) {
  return sizeof(SelShared) + sizeof(uint32_t) * (static_cast<size_t>(slice) + 2 * (static_cast<size_t>(slice) / 32));
}
static_assert(sel_smem(kEvictMaxSlots / kSelMaxCtas) <= 232448, "shared memory per CTA");

// Exclusive sum of v over the CTA's threads; *total gets the sum of all.
__device__ __forceinline__ uint32_t scan_cta(uint32_t v, uint32_t* warp_sum, uint32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  uint32_t w = warp_sum[lane], ws = w;   // kSelWarps == 32: every warp scans the warps' sums for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += y;
  }
  *total = __shfl_sync(0xffffffffu, ws, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, ws - w, warp);
  __syncthreads();
  return before + s - v;
}
static_assert(kSelWarps == 32, "scan_cta");

// One cluster of `cl` CTAs per request, each with a slice of its slots, whose keys stay in shared memory.  The m-th
// largest key is found by a radix selection of three digits (the CTAs' histograms are added up through
// distributed shared memory), ties are taken from the lowest slot on, and from the keep mask every staying
// token past slot m is written into a list in rank order, from which the free slots below m take theirs.
// Latency-bound: 7.6 us for 64 requests of 2112 or 4096 slots (one CTA each, of which the loads take
// 1.8, a digit 0.9, the mask 1.1 to 1.7, the outputs 1.3), 27 us for 4 requests of 131072 (eight CTAs each: loads
// and keys 6.3, digits 3.0 + 0.7 + 0.6 with 1.4 each for the exchange, mask 2, list 3.1, outputs 2.9; 16
// CTAs: 30 us, the exchange doubles).  Histograms are plain shared atomics: gathering equal digits of a warp first
// (__match_any_sync) took 11.5 us instead of 2.9, four copies changed nothing.
template <int cl>
__global__ void __launch_bounds__(kSelThreads, 1) mla_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint8_t sel_dyn[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_dyn);
  uint32_t* keys = reinterpret_cast<uint32_t*>(sel_dyn + sizeof(SelShared));
  const int log_slice = p.sel_log_slice, slice = 1 << log_slice, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint2* words_of = reinterpret_cast<uint2*>(keys + slice);   // 32 slots each: keep mask, kept slots before
  const int b = static_cast<int>(blockIdx.x) / cl;
  const uint32_t rank = cl > 1 ? cluster_ctarank() : 0;
  auto sync = [&] {
    if (cl > 1) cluster_sync();
    else __syncthreads();
  };
  for (int i = tid; i < 3 * kSelBins / 2; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.newest = -1;
  griddep_wait();
  griddep_launch_dependents();
  int n = p.seqlens[b];   // (new_seqlens may be the same array: not through the read-only path)
  if (n < 0 || n > p.slots) {
    if (tid == 0 && rank == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    n = 0;
  }
  const int m = min(n, p.budget);
  const float* w = p.weights + b * p.weights_stride;
  const int32_t* arr = p.arrival ? p.arrival + b * p.arrival_stride : nullptr;
  const int t0 = min(n, static_cast<int>(rank) << log_slice), count = min(n, t0 + slice) - t0;
  const int words = (count + 31) / 32;
  auto arrival_of = [&](int t) { return arr ? __ldg(arr + t) : t; };

  // e = 1 + the largest arrival number; four slots a load where both rows are 16-byte aligned
  int64_t e = n;
  const int step = arr && ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(arr)) & 15u) == 0 ? 4 : 1;
  if (arr) {
    __syncthreads();
    int top = -1;
    // the weights on their way into shared memory, each for the thread that uses it below
    for (int i = step * tid; i < count; i += step * kSelThreads) {
      if (step == 4 && i + 4 <= count) cp_async16(smem_u32(keys + i), w + t0 + i);
      else for (int j = i; j < min(count, i + step); ++j) cp_async4(keys + j, w + t0 + j);
    }
#pragma unroll 4
    for (int i = step * tid; i < count; i += step * kSelThreads) {
      if (step == 4 && i + 4 <= count) {
        const int4 a = __ldg(reinterpret_cast<const int4*>(arr + t0 + i));
        top = max(top, max(max(a.x, a.y), max(a.z, a.w)));
      } else {
        for (int j = i; j < min(count, i + step); ++j) top = max(top, __ldg(arr + t0 + j));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&sh.newest, top);
    sync();
    int newest = -1;
#pragma unroll
    for (int r = 0; r < cl; ++r)
      newest = max(newest, cl > 1 ? static_cast<int>(ld_cluster_u32(reinterpret_cast<uint32_t*>(&sh.newest), r)) : sh.newest);
    e = static_cast<int64_t>(newest) + 1;
    cp_async_wait_all();   // (where every token stays, too: nothing is on its way when the CTA leaves)
  }
  uint32_t cut = 0, ties = 0;   // keep key > cut, and the first `ties` slots with key == cut
  uint32_t tie_first = 0;       // ties in the CTAs before this one
  bool all_ties = true;         // every key == cut stays (distinct weights: no ranks among them are needed)
  if (m < n) {
    auto key = [&](int a, float weight) {
      return (a < p.sink || a >= e - p.recent) ? 0xffffffffu : weight_order(weight);
    };
#pragma unroll 4
    for (int i = step * tid; i < count; i += step * kSelThreads) {
      if (step == 4 && i + 4 <= count) {
        const int4 a = __ldg(reinterpret_cast<const int4*>(arr + t0 + i));
        uint4& k = *reinterpret_cast<uint4*>(keys + i);
        k = make_uint4(key(a.x, __uint_as_float(k.x)), key(a.y, __uint_as_float(k.y)), key(a.z, __uint_as_float(k.z)),
                       key(a.w, __uint_as_float(k.w)));
      } else {
        for (int j = i; j < min(count, i + step); ++j)
          keys[j] = key(arrival_of(t0 + j), arr ? __uint_as_float(keys[j]) : __ldg(w + t0 + j));
      }
    }
    uint32_t need = static_cast<uint32_t>(m);
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? kSelDigitBits : 32 - 2 * kSelDigitBits;
      const uint32_t high = pass == 0 ? 0u : ~0u << shift;   // the digits found so far
      shift -= bits;
      uint32_t* hist = sh.hist[pass];
      __syncthreads();   // (the first digit: keys and zeros are in place)
#pragma unroll 4
      for (int i = tid; i < count; i += kSelThreads) {
        const uint32_t k = keys[i];
        if (((k ^ cut) & high) == 0) {
          const uint32_t d = kSelBins - 1 - ((k >> shift) & ((1u << bits) - 1u));
          atomicAdd(&hist[d >> 1], 1u << (16 * (d & 1)));
        }
      }
      sync();
      // bins in descending order, two a thread
      uint32_t part[cl], bin[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < cl; ++r) part[r] = cl > 1 ? ld_cluster_u32(&hist[tid], r) : hist[tid];
#pragma unroll
      for (int r = 0; r < cl; ++r) bin[0] += part[r] & 0xffffu, bin[1] += part[r] >> 16;
      uint32_t all;
      uint32_t above = scan_cta(bin[0] + bin[1], sh.warp_sum, &all);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (above < need && need <= above + bin[j]) {
          sh.digit = static_cast<uint32_t>(kSelBins - 1 - (2 * tid + j));
          sh.need = need - above;
          sh.here = bin[j];
        }
        above += bin[j];
      }
      __syncthreads();
      cut |= sh.digit << shift;
      need = sh.need;
      if (need == sh.here) break;   // all of the digit's keys stay: key >= cut, whatever the digits further on
    }
    ties = need;
    all_ties = need == sh.here;
    if (cl > 1 && !all_ties) {
      const uint32_t d = kSelBins - 1 - (cut & ((1u << (32 - 2 * kSelDigitBits)) - 1u));
#pragma unroll
      for (int r = 0; r < cl; ++r) {
        const uint32_t k = ld_cluster_u32(&sh.hist[2][d >> 1], r) >> (16 * (d & 1)) & 0xffffu;
        tie_first += r < static_cast<int>(rank) ? k : 0u;
      }
    }
  }

  // keep mask: a warp walks a run of words; ties before the run are counted first
  const int run = (words + kSelWarps - 1) / kSelWarps;
  const int w0 = min(words, warp * run), w1 = min(words, w0 + run);
  uint32_t tie_rank = tie_first, all;
  if (!all_ties) {
    uint32_t mine = 0;
    for (int i = w0 * 32 + lane; i < w1 * 32; i += 32) mine += i < count && keys[i] == cut;
    tie_rank += scan_cta(mine, sh.warp_sum, &all);
    tie_rank = __shfl_sync(0xffffffffu, tie_rank, 0);   // that of the run's first lane: ties before the run
  }
  uint32_t kept = 0;
#pragma unroll 4
  for (int i = w0; i < w1; ++i) {
    const int t = i * 32 + lane;
    bool keep = t < count;
    if (m < n && all_ties) {
      keep = t < count && keys[t] >= cut;
    } else if (m < n) {
      const uint32_t k = t < count ? keys[t] : 0u;
      const bool tie = t < count && k == cut;
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      keep = t < count && (k > cut || (tie && tie_rank + __popc(tied & ((1u << lane) - 1u)) < ties));
      tie_rank += __popc(tied);
    }
    const uint32_t word = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) words_of[i] = make_uint2(word, kept);   // (before: within the run so far)
    kept += __popc(word);
  }
  const uint32_t before_run = __shfl_sync(0xffffffffu, scan_cta(lane == 0 ? kept : 0u, sh.warp_sum, &all), 0);
  for (int i = w0 + lane; i < w1; i += 32) words_of[i].y += before_run;
  __syncthreads();
  auto kept_before = [&](int t) {   // of this CTA's slots, below its slot t
    return t >= words * 32 ? all : words_of[t >> 5].y + __popc(words_of[t >> 5].x & ((1u << (t & 31)) - 1u));
  };
  const int m_here = max(0, min(count, m - t0));   // slots below m of this CTA
  if (tid == 0) sh.kept = all, sh.below = kept_before(m_here);
  sync();
  uint32_t first = 0, below = 0;   // kept slots of the CTAs before this one; kept slots below m
#pragma unroll
  for (int r = 0; r < cl; ++r) {
    const uint32_t k = cl > 1 ? ld_cluster_u32(&sh.kept, r) : 0u;
    first += r < static_cast<int>(rank) ? k : 0u;
    below += cl > 1 ? ld_cluster_u32(&sh.below, r) : sh.below;
  }
  // sources in rank order: entry i of the list lies in CTA i / slice (the keys are no longer needed)
#pragma unroll 4
  for (int i = (m_here / 32 + warp) * 32 + lane; i < words * 32; i += kSelThreads) {
    const uint2 word = words_of[i >> 5];
    const uint32_t lower = (1u << (i & 31)) - 1u;
    if (i >= m_here && (word.x & (lower + 1u))) {
      const uint32_t at = first + word.y + __popc(word.x & lower) - below;
      uint32_t* entry = keys + (at & (slice - 1));
      if (cl > 1) st_cluster_u32(map_to_rank(smem_u32(entry), at >> log_slice), static_cast<uint32_t>(t0 + i));
      else *entry = static_cast<uint32_t>(i);
    }
  }
  if (cl > 1) {
    __syncthreads();   // every thread has its words' counts; from here on they are the request's
    for (int i = tid; i < words; i += kSelThreads) words_of[i].y += first;
  }
  sync();

  // outputs, spread over the cluster, four slots a thread at a time (each is a chain of reads): slot j keeps its
  // token, or takes that of the next source
  constexpr int kEach = 4;
  const int64_t stride = static_cast<int64_t>(cl) * kSelThreads;
  for (int64_t j0 = static_cast<int64_t>(rank) * kSelThreads + tid; j0 < p.width; j0 += kEach * stride) {
    int src[kEach];
    uint2 word[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int64_t j = j0 + i * stride;
      src[i] = j < m ? static_cast<int>(j) : -1;
      const uint2* at = words_of + ((src[i] & (slice - 1)) >> 5);
      word[i] = src[i] < 0 ? make_uint2(~0u, 0) : cl > 1 ? ld_cluster_v2(at, src[i] >> log_slice) : *at;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint32_t bit = 1u << (src[i] & 31);
      if (!(word[i].x & bit)) {
        const uint32_t hole = static_cast<uint32_t>(src[i]) - word[i].y - __popc(word[i].x & (bit - 1u));
        src[i] = static_cast<int>(cl > 1 ? ld_cluster_u32(&keys[hole & (slice - 1)], hole >> log_slice) : keys[hole]);
      }
    }
    float weight[kEach];
    int number[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      weight[i] = src[i] >= 0 ? __ldg(w + src[i]) : 0.f;
      number[i] = src[i] >= 0 ? arrival_of(src[i]) : static_cast<int>(e + (j0 + i * stride - m));
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int64_t j = j0 + i * stride;
      if (j >= p.width) break;
      p.kept[b * p.width + j] = src[i];
      p.weights_out[b * p.width + j] = weight[i];
      if (p.arrival_out) p.arrival_out[b * p.width + j] = number[i];
    }
  }
  if (cl > 1) cluster_done();   // no CTA leaves while another reads its shared memory
  if (tid == 0 && rank == 0) p.new_seqlens[b] = m;   // last: it may be the array that the lengths came from
}

// Copies the rows of moved tokens: 16-byte units, two rows in flight a warp.  A warp takes kMoveSlots slots; sources
// lie at or past the new length and targets below it, so no row is both.  HBM-bound: 64 requests, 4096 -> 2048 slots
// (65 thousand rows, 151 MB read and written) 24.2 us, 6.2 TB/s.  With 16 slots a warp 25.5, its 1024 blocks being one
// uneven wave; with 8 as with 12, but 0.3 us more where few rows move.  Rows as one run of units, nine full loads a lane
// in flight: 0.7 us less here, 1 to 2 more where few rows move and for FP8.
template <int kRowBytes>
__global__ void __launch_bounds__(256) mla_evict_move_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kUnits = kRowBytes / 16, kEach = (kUnits + 31) / 32;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t j = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kMoveSlots + lane;
  const int top = min(p.budget, p.slots);
  int src = -1;
  if (lane < kMoveSlots && j < top) src = p.kept[b * p.width + j];
  auto row_of = [&](int t) -> int64_t {
    const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + t / kPageTokens);
    return blk >= 0 && blk < p.num_blocks ? static_cast<int64_t>(blk) * kPageTokens + t % kPageTokens : -1;
  };
  int64_t from = -1, to = -1;
  if (src >= 0 && src != j) {
    from = row_of(src);
    to = row_of(static_cast<int>(j));
    if (from < 0 || to < 0) {
      atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
      from = -1;
    }
  }
  uint32_t todo = __ballot_sync(0xffffffffu, from >= 0);
  uint8_t* kv = static_cast<uint8_t*>(p.kv);
  while (todo) {
    uint4 v[2][kEach];
    int64_t t[2];
    bool have[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      have[r] = todo != 0;
      const int l = have[r] ? __ffs(todo) - 1 : 0;
      todo &= todo - 1;
      const int64_t f = __shfl_sync(0xffffffffu, from, l);
      t[r] = __shfl_sync(0xffffffffu, to, l);
#pragma unroll
      for (int u = 0; u < kEach; ++u)
        if (have[r] && u * 32 + lane < kUnits) v[r][u] = *reinterpret_cast<const uint4*>(kv + f * kRowBytes + (u * 32 + lane) * 16);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int u = 0; u < kEach; ++u)
        if (have[r] && u * 32 + lane < kUnits) *reinterpret_cast<uint4*>(kv + t[r] * kRowBytes + (u * 32 + lane) * 16) = v[r][u];
  }
}

// ------------------------------------------------------------------- host --
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks the rotation's arguments and fills the table; false where they are invalid.
bool rope_table(const int32_t* sections, int n_axes, int interleaved, float theta, RopeTable* t) {
  if (!sections || n_axes < 1 || n_axes > kRopeMaxAxes || !std::isfinite(theta) || !(theta > 1.f)) return false;
  int left[kRopeMaxAxes], sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0 || sections[a] > kPairs) return false;
    left[a] = sections[a];
    sum += sections[a];
  }
  if (sum != kPairs) return false;
  for (int j = 0, a = 0; j < kPairs;) {
    if (left[a] > 0) {
      --left[a];
      t->axis[j++] = static_cast<uint8_t>(a);
      if (interleaved) a = (a + 1) % n_axes;
    } else {
      a = (a + 1) % n_axes;
    }
  }
  // theta is a constant of the model: its 32 powers are kept from the thread's last call with the same one
  thread_local float kept_theta = 0.f;
  thread_local float kept[2][kPairs];
  if (kept_theta != theta) {
    for (int j = 0; j < kPairs; ++j) {
      const double inv = std::pow(static_cast<double>(theta), -2.0 * j / 64.0);
      kept[0][j] = static_cast<float>(inv);
      kept[1][j] = static_cast<float>(inv - static_cast<double>(kept[0][j]));
    }
    kept_theta = theta;
  }
  std::memcpy(t->hi, kept[0], sizeof(t->hi));
  std::memcpy(t->lo, kept[1], sizeof(t->lo));
  const double two_pi = 6.283185307179586476925286766559;
  t->two_pi_hi = static_cast<float>(two_pi);
  t->two_pi_lo = static_cast<float>(two_pi - static_cast<double>(t->two_pi_hi));
  return true;
}

enum class CacheFormat { kBf16, kFp8, kFp4 };

mla_status_t append_impl(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe, int64_t k_pe_row_stride,
                         void* kv_cache, CacheFormat format, float kv_scale, int64_t num_blocks,
                         const int32_t* block_table, int max_blocks, const int32_t* seqlens, const int32_t* new_offsets,
                         int N, int B, const int32_t* positions, int64_t positions_stride, const int32_t* sections,
                         int n_axes, int interleaved, float rope_theta, mla_stream_t stream,
                         const mla_bf16_t* norm_weight = nullptr, float norm_eps = 0.f) {
  const bool fp8 = format == CacheFormat::kFp8, fp4 = format == CacheFormat::kFp4;
  if (!c || !k_pe || !kv_cache || !block_table || !seqlens || N < 1 || B < 1 || num_blocks < 1 || max_blocks < 1)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(c, 16) || !aligned(k_pe, 16) || !aligned(kv_cache, 16) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(new_offsets, 4) || !aligned(positions, 4))
    return MLA_ERR_INVALID_ARG;
  if (c_row_stride < kDimV || c_row_stride % 8 || k_pe_row_stride < 64 || k_pe_row_stride % 8)
    return MLA_ERR_INVALID_ARG;
  if (!new_offsets && N % B) return MLA_ERR_INVALID_ARG;
  if ((fp8 || fp4) && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  if (fp4 && !fp4_scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  if (norm_weight && (!aligned(norm_weight, 16) || !std::isfinite(norm_eps) || !(norm_eps >= 0.f))) return MLA_ERR_INVALID_ARG;
  AppendParams p = {};
  if (positions && (positions_stride < N || !rope_table(sections, n_axes, interleaved, rope_theta, &p.table)))
    return MLA_ERR_INVALID_ARG;
  if (num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens || B > kScheduleMaxB || N > kMaxRows)
    return MLA_ERR_UNSUPPORTED;
  p.c = reinterpret_cast<const __nv_bfloat16*>(c);
  p.pe = reinterpret_cast<const __nv_bfloat16*>(k_pe);
  p.c_row = c_row_stride;
  p.pe_row = k_pe_row_stride;
  p.kv = kv_cache;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.offsets = new_offsets;
  p.N = N;
  p.B = B;
  p.rows_each = N / B;
  p.positions = positions;
  p.pos_stride = positions_stride;
  p.kv_scale = kv_scale;
  p.kv_inv = 1.f / kv_scale;
  int exponent = 0;
  const bool divide = std::frexp(kv_scale, &exponent) != 0.5f || !std::isnormal(p.kv_inv);   // no power of two
  p.norm = reinterpret_cast<const __nv_bfloat16*>(norm_weight);
  p.norm_eps = norm_eps;
  p.status = device_status_word();
  if (!p.status) return MLA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>((N + 3) / 4)), dim3(128), 0,
                                            reinterpret_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = fp4      ? (norm_weight ? cudaLaunchKernelEx(&cfg, mla_append_fp4_kernel<true>, p)
                                                : cudaLaunchKernelEx(&cfg, mla_append_fp4_kernel<false>, p))
                        : !fp8   ? cudaLaunchKernelEx(&cfg, mla_append_kernel<false, false>, p)
                        : divide ? cudaLaunchKernelEx(&cfg, mla_append_kernel<true, true>, p)
                                 : cudaLaunchKernelEx(&cfg, mla_append_kernel<true, false>, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

bool overlap(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

mla_status_t evict_impl(void* kv_cache, bool fp8, int64_t num_blocks, const int32_t* block_table, int max_blocks,
                        const int32_t* seqlens, int B, const float* weights, int64_t weights_stride,
                        const int32_t* arrival, int64_t arrival_stride, int budget, int sink, int recent,
                        int32_t* new_seqlens, int32_t* kept, float* weights_out, int32_t* arrival_out, int64_t width,
                        mla_stream_t stream) {
  if (!kv_cache || !block_table || !seqlens || !weights || !new_seqlens || !kept || !weights_out)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(seqlens, 4) || !aligned(weights, 4) ||
      !aligned(arrival, 4) || !aligned(new_seqlens, 4) || !aligned(kept, 4) || !aligned(weights_out, 4) ||
      !aligned(arrival_out, 4))
    return MLA_ERR_INVALID_ARG;
  if (B < 1 || num_blocks < 1 || max_blocks < 1 || weights_stride < 1 || (arrival && arrival_stride < 1) || width < 1)
    return MLA_ERR_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget) return MLA_ERR_INVALID_ARG;
  int64_t slots = static_cast<int64_t>(max_blocks) * kPageTokens;
  slots = slots < weights_stride ? slots : weights_stride;
  if (width < (budget < slots ? budget : slots)) return MLA_ERR_INVALID_ARG;
  if (slots > kEvictMaxSlots || num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens || B > kScheduleMaxB)
    return MLA_ERR_UNSUPPORTED;
  if (arrival && arrival_stride < slots) slots = arrival_stride;   // what is read of a row
  // what is written may overlap neither what is read nor one another (new_seqlens may be seqlens)
  const uint64_t out_bytes = static_cast<uint64_t>(B) * width * 4, rows = static_cast<uint64_t>(B) - 1;
  const struct { const void* at; uint64_t bytes; } span[] = {
      {kept, out_bytes}, {weights_out, out_bytes}, {arrival_out, out_bytes}, {new_seqlens, (rows + 1) * 4},
      {new_seqlens == seqlens ? nullptr : seqlens, (rows + 1) * 4}, {block_table, (rows + 1) * max_blocks * 4},
      {weights, (rows * weights_stride + slots) * 4}, {arrival, (rows * arrival_stride + slots) * 4}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (span[i].at && span[j].at && overlap(span[i].at, span[i].bytes, span[j].at, span[j].bytes))
        return MLA_ERR_INVALID_ARG;
  EvictParams p = {};
  p.kv = kv_cache;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.arrival = arrival;
  p.arrival_stride = arrival_stride;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.slots = static_cast<int>(slots);
  p.new_seqlens = new_seqlens;
  p.kept = kept;
  p.weights_out = weights_out;
  p.arrival_out = arrival_out;
  p.width = width;
  p.status = device_status_word();
  if (!p.status) return MLA_ERR_CUDA;
  int cl = 1;
  while (cl < kSelMaxCtas && static_cast<int64_t>(cl) * kSelSlotsPerCta < slots) cl *= 2;
  p.sel_log_slice = 5;
  while (static_cast<int64_t>(cl) << p.sel_log_slice < slots) ++p.sel_log_slice;
  const size_t smem = sel_smem(1 << p.sel_log_slice);
  const auto select = cl == 1 ? mla_evict_select_kernel<1> : cl == 2 ? mla_evict_select_kernel<2>
                      : cl == 4 ? mla_evict_select_kernel<4> : mla_evict_select_kernel<8>;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sel_smem(kEvictMaxSlots / kSelMaxCtas))) != cudaSuccess)
    return MLA_ERR_CUDA;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t sel = pdl_config(dim3(static_cast<unsigned>(B * cl)), dim3(kSelThreads), smem, cs, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  sel.numAttrs = cl > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&sel, select, p) != cudaSuccess) return MLA_ERR_CUDA;
  const int64_t top = budget < slots ? budget : slots;
  constexpr int kMoveBlock = 8 * kMoveSlots;   // slots of a block's 8 warps
  const cudaLaunchConfig_t mv = pdl_config(dim3(static_cast<unsigned>((top + kMoveBlock - 1) / kMoveBlock), static_cast<unsigned>(B)),
                                           dim3(256), 0, cs, attr);
  const cudaError_t e = fp8 ? cudaLaunchKernelEx(&mv, mla_evict_move_kernel<kDimQK>, p)
                            : cudaLaunchKernelEx(&mv, mla_evict_move_kernel<kDimQK * 2>, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_rope_axes(const mla_bf16_t* x, int64_t x_row_stride, int64_t x_head_stride, mla_bf16_t* out,
                           int64_t out_row_stride, int64_t out_head_stride, const int32_t* positions,
                           int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                           float rope_theta, int inverse, int N, int H, mla_stream_t stream) {
  if (!x || !out || !positions || N < 1 || H < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || positions_stride < N) return MLA_ERR_INVALID_ARG;
  if (x_row_stride % 8 || x_head_stride % 8 || out_row_stride % 8 || out_head_stride % 8) return MLA_ERR_INVALID_ARG;
  // every row of out is written once: heads and tokens may not fall on one another
  auto spread = [&](int64_t row, int64_t head) {
    if (row < 0 || head < 0) return false;
    if (H > 1 && head < 64) return false;
    if (N == 1) return true;
    const int64_t heads = H > 1 ? static_cast<int64_t>(H - 1) * head + 64 : 64;
    const int64_t rows = static_cast<int64_t>(N - 1) * row + 64;
    return row >= heads || (H > 1 && row >= 64 && head >= rows);
  };
  if (x_row_stride < 0 || x_head_stride < 0 || !spread(out_row_stride, out_head_stride)) return MLA_ERR_INVALID_ARG;
  RopeParams p = {};
  if (!rope_table(sections, n_axes, interleaved, rope_theta, &p.table)) return MLA_ERR_INVALID_ARG;
  if (N > kMaxRows || H > 65535 * 32) return MLA_ERR_UNSUPPORTED;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.x_row = x_row_stride;
  p.x_head = x_head_stride;
  p.out_row = out_row_stride;
  p.out_head = out_head_stride;
  p.positions = positions;
  p.pos_stride = positions_stride;
  p.N = N;
  p.H = H;
  p.sign = inverse ? -1.f : 1.f;
  if (!device_status_word()) return MLA_ERR_CUDA;
  while ((1 << p.log_heads) < (H < 32 ? H : 32)) ++p.log_heads;
  const int tokens = 32 >> p.log_heads;
  const int64_t blocks = (static_cast<int64_t>(N) + tokens - 1) / tokens;
  // four rounds of heads a block where that still leaves every SM several blocks; else a round each, which spreads
  // few tokens over the GPU
  const int rounds = H > 32 && blocks * ((H + 127) / 128) >= 4 * 152 ? 4 : 1;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(
      dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((H + 32 * rounds - 1) / (32 * rounds))), dim3(256), 0,
      reinterpret_cast<cudaStream_t>(stream), attr);
  return (rounds == 4 ? cudaLaunchKernelEx(&cfg, mla_rope_axes_kernel<4>, p)
                      : cudaLaunchKernelEx(&cfg, mla_rope_axes_kernel<1>, p)) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

mla_status_t mla_cache_append(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe,
                              int64_t k_pe_row_stride, mla_bf16_t* kv_cache, int64_t num_blocks,
                              const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                              const int32_t* new_offsets, int N, int B, const int32_t* positions,
                              int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                              float rope_theta, mla_stream_t stream) {
  return append_impl(c, c_row_stride, k_pe, k_pe_row_stride, kv_cache, CacheFormat::kBf16, 1.f, num_blocks, block_table, max_blocks,
                     seqlens, new_offsets, N, B, positions, positions_stride, sections, n_axes, interleaved, rope_theta,
                     stream);
}

mla_status_t mla_cache_append_fp8(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe,
                                  int64_t k_pe_row_stride, uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                                  const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                  const int32_t* new_offsets, int N, int B, const int32_t* positions,
                                  int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                                  float rope_theta, mla_stream_t stream) {
  return append_impl(c, c_row_stride, k_pe, k_pe_row_stride, kv_cache, CacheFormat::kFp8, kv_scale, num_blocks,
                     block_table, max_blocks, seqlens, new_offsets, N, B, positions, positions_stride, sections, n_axes,
                     interleaved, rope_theta, stream);
}

mla_status_t mla_cache_append_fp4(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe,
                                  int64_t k_pe_row_stride, uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                                  const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                  const int32_t* new_offsets, int N, int B, const int32_t* positions,
                                  int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                                  float rope_theta, const mla_bf16_t* norm_weight, float norm_eps, mla_stream_t stream) {
  return append_impl(c, c_row_stride, k_pe, k_pe_row_stride, kv_cache, CacheFormat::kFp4, kv_scale, num_blocks,
                     block_table, max_blocks, seqlens, new_offsets, N, B, positions, positions_stride, sections, n_axes,
                     interleaved, rope_theta, stream, norm_weight, norm_eps);
}

mla_status_t mla_evict(mla_bf16_t* kv_cache, int64_t num_blocks, const int32_t* block_table, int max_blocks,
                       const int32_t* seqlens, int B, const float* weights, int64_t weights_stride,
                       const int32_t* arrival, int64_t arrival_stride, int budget, int sink, int recent,
                       int32_t* new_seqlens, int32_t* kept, float* weights_out, int32_t* arrival_out, int64_t width,
                       mla_stream_t stream) {
  return evict_impl(kv_cache, false, num_blocks, block_table, max_blocks, seqlens, B, weights, weights_stride, arrival,
                    arrival_stride, budget, sink, recent, new_seqlens, kept, weights_out, arrival_out, width, stream);
}

mla_status_t mla_evict_fp8(uint8_t* kv_cache, int64_t num_blocks, const int32_t* block_table, int max_blocks,
                           const int32_t* seqlens, int B, const float* weights, int64_t weights_stride,
                           const int32_t* arrival, int64_t arrival_stride, int budget, int sink, int recent,
                           int32_t* new_seqlens, int32_t* kept, float* weights_out, int32_t* arrival_out,
                           int64_t width, mla_stream_t stream) {
  return evict_impl(kv_cache, true, num_blocks, block_table, max_blocks, seqlens, B, weights, weights_stride, arrival,
                    arrival_stride, budget, sink, recent, new_seqlens, kept, weights_out, arrival_out, width, stream);
}

}  // extern "C"
