// The latent cache over a request's life: RoPE with several position axes, the write of
// new rows into the paged cache (bf16 or E4M3), and eviction by accumulated attention
// weight.  C entries at the end (declared in mla.h).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr int kRopeMaxAxes = 4;
constexpr int kPairs = 32;              // rotated pairs of a 64-value row

// Inverse frequencies theta^(-2j/64) and 2*pi as float pairs (hi + lo), and each pair's axis.
struct RopeTable {
  float hi[kPairs], lo[kPairs];
  float two_pi_hi, two_pi_lo;
  uint8_t axis[kPairs];
};

// cos and sin of pair j's angle at `pos`: the arithmetic of rope_row (mla_rope.cuh), whose
// argument reduction keeps the angle within ~1e-7 rad for |pos| < 2^24.
__device__ __forceinline__ float2 rope_turn(const RopeTable& t, int j, int pos) {
  const float fp = static_cast<float>(pos);
  const float inv_two_pi = 1.0f / t.two_pi_hi;
  const float a_hi = fp * t.hi[j];
  const float a_lo = fmaf(fp, t.lo[j], fmaf(fp, t.hi[j], -a_hi));
  const float k = rintf(a_hi * inv_two_pi);
  const float r = fmaf(-k, t.two_pi_lo, fmaf(-k, t.two_pi_hi, a_hi)) + a_lo;
  float sn, cs;
  __sincosf(r, &sn, &cs);   // |r| <= pi + 1e-6: the hardware sine/cosine, absolute error < 2^-21
  return make_float2(cs, sn);
}

// ------------------------------------------------------------------- rope --
struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t x_row, x_head, out_row, out_head;
  const int32_t* positions;
  int64_t pos_stride;
  int N, H;
  float sign;               // -1: the inverse rotation
  RopeTable table;
};

// One block per token and 32 heads; a thread turns 4 pairs (16 bytes) of one head.
__global__ void __launch_bounds__(256) mla_rope_axes_kernel(const __grid_constant__ RopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x;
  const int u = threadIdx.x & 7;                       // 16-byte unit of the row: pairs 4u .. 4u + 3
  const int h = blockIdx.y * 32 + (threadIdx.x >> 3);
  if (h >= p.H) return;
  const uint4 v = *reinterpret_cast<const uint4*>(p.x + n * p.x_row + h * p.x_head + u * 8);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * u + i;
    const float2 t = rope_turn(p.table, j, __ldg(p.positions + p.table.axis[j] * p.pos_stride + n));
    const float cs = t.x, sn = t.y * p.sign;
    const float x0 = bf16_lo(w[i]), x1 = bf16_hi(w[i]);
    w[i] = pack_bf16x2(fmaf(x0, cs, -x1 * sn), fmaf(x0, sn, x1 * cs));
  }
  *reinterpret_cast<uint4*>(p.out + n * p.out_row + h * p.out_head + u * 8) = make_uint4(w[0], w[1], w[2], w[3]);
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
  float kv_scale;
  int* status;
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

// One warp per new row: 72 units of 8 values, lane l takes units l, l + 32 and (l < 8) the
// rotated unit 64 + l.
template <bool F8>
__global__ void __launch_bounds__(128) mla_append_kernel(const __grid_constant__ AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= p.N) return;
  int b, end;
  if (p.offsets != nullptr) {
    b = request_of(p.offsets, p.B, r, lane);
    if (b < 0 || b >= p.B) return;
    end = __ldg(p.offsets + b + 1);
  } else {
    b = r / p.rows_each;
    end = (b + 1) * p.rows_each;
  }
  const int64_t t = static_cast<int64_t>(__ldg(p.seqlens + b)) - (end - r);
  int64_t row = -1;
  if (t >= 0 && t < static_cast<int64_t>(p.max_blocks) * kPageTokens) {
    const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + t / kPageTokens);
    if (blk >= 0 && blk < p.num_blocks) row = static_cast<int64_t>(blk) * kPageTokens + t % kPageTokens;
  }
  if (row < 0) {
    if (lane == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    return;
  }
  auto store = [&](int u, const float (&f)[8]) {
    if constexpr (F8) {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = cvt_e4m3x2(__fdiv_rn(f[4 * i], p.kv_scale), __fdiv_rn(f[4 * i + 1], p.kv_scale)) |
               (cvt_e4m3x2(__fdiv_rn(f[4 * i + 2], p.kv_scale), __fdiv_rn(f[4 * i + 3], p.kv_scale)) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kv) + row * kDimQK + u * 8) = make_uint2(w[0], w[1]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.kv) + row * kDimQK + u * 8) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  auto widen = [](const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
  };
  const uint4* c = reinterpret_cast<const uint4*>(p.c + r * p.c_row);
  float f[8];
  const uint4 c0 = __ldg(c + lane), c1 = __ldg(c + 32 + lane);
  if (lane < 8) {
    const uint4 e = __ldg(reinterpret_cast<const uint4*>(p.pe + r * p.pe_row) + lane);
    widen(e, f);
    if (p.positions != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * lane + i;
        const float2 turn = rope_turn(p.table, j, __ldg(p.positions + p.table.axis[j] * p.pos_stride + r));
        const float x0 = f[2 * i], x1 = f[2 * i + 1];
        f[2 * i] = fmaf(x0, turn.x, -x1 * turn.y);
        f[2 * i + 1] = fmaf(x0, turn.y, x1 * turn.x);
      }
    }
    store(64 + lane, f);
  }
  widen(c0, f);
  store(lane, f);
  widen(c1, f);
  store(32 + lane, f);
}

// ------------------------------------------------------------------ evict --
constexpr int kEvictMaxSlots = 524288;  // a request's keep mask and its prefix counts fit shared memory
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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

// One block per request.  The m-th largest key is found by a radix selection (four passes of 8
// bits over the keys), ties are taken from the lowest slot on, and the keep mask and its prefix
// counts (one bit and 1/32 word a slot, in shared memory) give every free slot its source.
__global__ void __launch_bounds__(kSelThreads) mla_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t sel_smem[];          // mask [words], then prefix [words + 1]
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sum[kSelWarps + 1];
  __shared__ uint32_t s_key, s_left;
  __shared__ int s_max;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int n = p.seqlens[b];   // (new_seqlens may be the same array: not through the read-only path)
  if (n < 0 || n > p.slots) {
    if (tid == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    n = 0;
  }
  const int m = min(n, p.budget);
  const float* w = p.weights + b * p.weights_stride;
  const int32_t* arr = p.arrival ? p.arrival + b * p.arrival_stride : nullptr;
  const int words = (n + 31) / 32;
  uint32_t* mask = sel_smem;
  uint32_t* prefix = sel_smem + (p.slots + 31) / 32;
  auto arrival_of = [&](int t) { return arr ? __ldg(arr + t) : t; };

  // e = 1 + the largest arrival number
  if (tid == 0) s_max = -1;
  __syncthreads();
  if (arr) {
    int top = -1;
    for (int t = tid; t < n; t += kSelThreads) top = max(top, __ldg(arr + t));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&s_max, top);
  } else if (tid == 0) {
    s_max = n - 1;
  }
  __syncthreads();
  const int64_t e = static_cast<int64_t>(s_max) + 1;
  auto key_of = [&](int t) {
    const int a = arrival_of(t);
    return (a < p.sink || a >= e - p.recent) ? 0xffffffffu : weight_order(__ldg(w + t));
  };

  uint32_t cut = 0, ties = 0;   // keep key > cut, and the first `ties` slots with key == cut
  if (m < n) {
    uint32_t left = static_cast<uint32_t>(m);
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int t = tid; t < n; t += kSelThreads) {
        const uint32_t k = key_of(t);
        if (((k ^ cut) & high) == 0) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {   // the digit in which the m-th largest key lies
        uint32_t need = left;
        int d = 255;
        while (d > 0 && hist[d] < need) need -= hist[d--];
        s_key = cut | (static_cast<uint32_t>(d) << shift);
        s_left = need;
      }
      __syncthreads();
      cut = s_key;
      left = s_left;
    }
    ties = left;
  }

  // keep mask: each warp walks a run of words; ties before its run are counted first
  const int run = (words + kSelWarps - 1) / kSelWarps;
  const int w0 = min(words, warp * run), w1 = min(words, w0 + run);
  auto scan_warps = [&](uint32_t v) {   // exclusive sum over the warps of lane 0's v; total in warp_sum[kSelWarps]
    if (lane == 0) warp_sum[warp] = v;
    __syncthreads();
    if (warp == 0) {
      const uint32_t x = warp_sum[lane];
      uint32_t s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      warp_sum[lane] = s - x;
      if (lane == 31) warp_sum[kSelWarps] = s;
    }
    __syncthreads();
    const uint32_t r = warp_sum[warp];
    __syncthreads();
    return r;
  };
  uint32_t tie_rank = 0;
  if (m < n) {
    uint32_t mine = 0;
    for (int i = w0; i < w1; ++i) {
      const int t = i * 32 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, t < n && key_of(t) == cut));
    }
    tie_rank = scan_warps(mine);
  }
  uint32_t kept_mine = 0;
  for (int i = w0; i < w1; ++i) {
    const int t = i * 32 + lane;
    bool keep = t < n;
    if (m < n) {
      const uint32_t k = t < n ? key_of(t) : 0u;
      const bool tie = t < n && k == cut;
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      keep = t < n && (k > cut || (tie && tie_rank + __popc(tied & ((1u << lane) - 1u)) < ties));
      tie_rank += __popc(tied);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) {
      mask[i] = bits;
      prefix[i] = kept_mine;   // within the warp's run
    }
    kept_mine += __popc(bits);
  }
  const uint32_t before = scan_warps(kept_mine);
  for (int i = w0 + lane; i < w1; i += 32) prefix[i] += before;
  __syncthreads();

  // outputs: slot j keeps its token, or takes that of the next source
  auto kept_before = [&](int t) {   // kept slots below t
    return t >= words * 32 ? static_cast<uint32_t>(m) : prefix[t >> 5] + __popc(mask[t >> 5] & ((1u << (t & 31)) - 1u));
  };
  const uint32_t below = kept_before(m);
  for (int64_t j = tid; j < p.width; j += kSelThreads) {
    int src = -1;
    if (j < m) {
      const int t = static_cast<int>(j);
      src = t;
      if (!((mask[t >> 5] >> (t & 31)) & 1u)) {
        const uint32_t rank = below + (static_cast<uint32_t>(t) - kept_before(t));   // the rank-th kept slot
        int lo = m >> 5, hi = words - 1;   // the last word with prefix <= rank
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (prefix[mid] <= rank) lo = mid; else hi = mid - 1;
        }
        src = lo * 32 + static_cast<int>(__fns(mask[lo], 0, static_cast<int>(rank - prefix[lo]) + 1));
      }
    }
    const int64_t at = b * p.width + j;
    p.kept[at] = src;
    p.weights_out[at] = src >= 0 ? __ldg(w + src) : 0.f;
    if (p.arrival_out) p.arrival_out[at] = src >= 0 ? arrival_of(src) : static_cast<int32_t>(e + (j - m));
  }
  if (tid == 0) p.new_seqlens[b] = m;   // last: it may be the array that the lengths came from
}

// Copies the rows of moved tokens.  A warp takes 32 slots; sources lie at or past the new length
// and targets below it, so no row is both.
template <int kRowBytes>
__global__ void __launch_bounds__(256) mla_evict_move_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kUnits = kRowBytes / 16;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t j = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 32 + lane;
  const int top = min(p.budget, p.slots);
  int src = -1;
  if (j < top) src = p.kept[b * p.width + j];
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
  while (todo) {
    const int l = __ffs(todo) - 1;
    todo &= todo - 1;
    const int64_t f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, to, l);
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.kv) + f * kRowBytes);
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.kv) + t * kRowBytes);
    for (int u = lane; u < kUnits; u += 32) d[u] = s[u];
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
  for (int j = 0; j < kPairs; ++j) {
    const double inv = std::pow(static_cast<double>(theta), -2.0 * j / 64.0);
    t->hi[j] = static_cast<float>(inv);
    t->lo[j] = static_cast<float>(inv - static_cast<double>(t->hi[j]));
  }
  const double two_pi = 6.283185307179586476925286766559;
  t->two_pi_hi = static_cast<float>(two_pi);
  t->two_pi_lo = static_cast<float>(two_pi - static_cast<double>(t->two_pi_hi));
  return true;
}

mla_status_t append_impl(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe, int64_t k_pe_row_stride,
                         void* kv_cache, bool fp8, float kv_scale, int64_t num_blocks, const int32_t* block_table,
                         int max_blocks, const int32_t* seqlens, const int32_t* new_offsets, int N, int B,
                         const int32_t* positions, int64_t positions_stride, const int32_t* sections, int n_axes,
                         int interleaved, float rope_theta, mla_stream_t stream) {
  if (!c || !k_pe || !kv_cache || !block_table || !seqlens || N < 1 || B < 1 || num_blocks < 1 || max_blocks < 1)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(c, 16) || !aligned(k_pe, 16) || !aligned(kv_cache, 16) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(new_offsets, 4) || !aligned(positions, 4))
    return MLA_ERR_INVALID_ARG;
  if (c_row_stride < kDimV || c_row_stride % 8 || k_pe_row_stride < 64 || k_pe_row_stride % 8)
    return MLA_ERR_INVALID_ARG;
  if (!new_offsets && N % B) return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  AppendParams p = {};
  if (positions && (positions_stride < N || !rope_table(sections, n_axes, interleaved, rope_theta, &p.table)))
    return MLA_ERR_INVALID_ARG;
  if (num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens || B > kScheduleMaxB) return MLA_ERR_UNSUPPORTED;
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
  p.status = device_status_word();
  if (!p.status) return MLA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>((N + 3) / 4)), dim3(128), 0,
                                            reinterpret_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = fp8 ? cudaLaunchKernelEx(&cfg, mla_append_kernel<true>, p)
                            : cudaLaunchKernelEx(&cfg, mla_append_kernel<false>, p);
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
  const uint64_t in_w = (static_cast<uint64_t>(B) - 1) * weights_stride + slots;
  const uint64_t out = static_cast<uint64_t>(B) * width;
  const uint64_t in_a = arrival ? (static_cast<uint64_t>(B) - 1) * arrival_stride + slots : 0;
  for (const void* o : {static_cast<const void*>(weights_out), static_cast<const void*>(arrival_out)})
    if (o && (overlap(o, out * 4, weights, in_w * 4) || (arrival && overlap(o, out * 4, arrival, in_a * 4))))
      return MLA_ERR_INVALID_ARG;
  if (slots > kEvictMaxSlots || num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens || B > kScheduleMaxB)
    return MLA_ERR_UNSUPPORTED;
  if (arrival && arrival_stride < slots) slots = arrival_stride;
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
  const size_t smem = (2 * ((static_cast<size_t>(slots) + 31) / 32) + 1) * sizeof(uint32_t);
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(mla_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>((2 * (kEvictMaxSlots / 32) + 1) * sizeof(uint32_t))) != cudaSuccess)
    return MLA_ERR_CUDA;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t sel = pdl_config(dim3(static_cast<unsigned>(B)), dim3(kSelThreads), smem, cs, attr);
  if (cudaLaunchKernelEx(&sel, mla_evict_select_kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  const int64_t top = budget < slots ? budget : slots;
  const cudaLaunchConfig_t mv =
      pdl_config(dim3(static_cast<unsigned>((top + 255) / 256), static_cast<unsigned>(B)), dim3(256), 0, cs, attr);
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
  if (H > 65535 * 32) return MLA_ERR_UNSUPPORTED;
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
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(static_cast<unsigned>(N), static_cast<unsigned>((H + 31) / 32)), dim3(256), 0,
                 reinterpret_cast<cudaStream_t>(stream), attr);
  return cudaLaunchKernelEx(&cfg, mla_rope_axes_kernel, p) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status_t mla_cache_append(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe,
                              int64_t k_pe_row_stride, mla_bf16_t* kv_cache, int64_t num_blocks,
                              const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                              const int32_t* new_offsets, int N, int B, const int32_t* positions,
                              int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                              float rope_theta, mla_stream_t stream) {
  return append_impl(c, c_row_stride, k_pe, k_pe_row_stride, kv_cache, false, 1.f, num_blocks, block_table, max_blocks,
                     seqlens, new_offsets, N, B, positions, positions_stride, sections, n_axes, interleaved, rope_theta,
                     stream);
}

mla_status_t mla_cache_append_fp8(const mla_bf16_t* c, int64_t c_row_stride, const mla_bf16_t* k_pe,
                                  int64_t k_pe_row_stride, uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                                  const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                  const int32_t* new_offsets, int N, int B, const int32_t* positions,
                                  int64_t positions_stride, const int32_t* sections, int n_axes, int interleaved,
                                  float rope_theta, mla_stream_t stream) {
  return append_impl(c, c_row_stride, k_pe, k_pe_row_stride, kv_cache, true, kv_scale, num_blocks, block_table,
                     max_blocks, seqlens, new_offsets, N, B, positions, positions_stride, sections, n_axes, interleaved,
                     rope_theta, stream);
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
