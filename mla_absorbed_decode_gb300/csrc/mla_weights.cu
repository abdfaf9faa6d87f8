// Attention weight of every cached token: weights[b, t] += sum over the request's query rows of
// exp(scale * <q, kv_t> - lse).  C entries at the end (declared in mla.h).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

struct WeightsParams {
  const __nv_bfloat16* q;
  const float* lse;
  const void* kv;
  float kv_scale;
  int64_t num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seqlens;
  int B, s_q, H, rows, causal;
  int slots;                 // largest length: min(64 max_blocks, weights_stride)
  float scale_hi, scale_lo;  // softmax_scale * log2(e) (times kv_scale) as a float pair
  float* weights;
  int64_t weights_stride;
  int* status;
};

// One block per page and request; a warp takes 8 tokens of the page, lane l dims 18 l .. 18 l + 17.
template <bool F8>
__global__ void __launch_bounds__(256) mla_attn_weights_kernel(const WeightsParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, page = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = __ldg(p.seqlens + b);
  if (n < 0 || n > p.slots) {
    if (page == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    return;
  }
  if (page * kPageTokens >= n) return;
  const int blk = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + page);
  if (blk < 0 || blk >= p.num_blocks) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
    return;
  }
  for (int i = warp; i < kPageTokens; i += 8) {
    const int t = page * kPageTokens + i;
    if (t >= n) break;
    const int64_t at = (static_cast<int64_t>(blk) * kPageTokens + i) * kDimQK + lane * 18;
    float k[18];
#pragma unroll
    for (int d = 0; d < 9; ++d) {
      if constexpr (F8) {
        const uint32_t v = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.kv) + at + 2 * d);
        const float2 f = e4m3x2_to_float2(v);
        k[2 * d] = f.x, k[2 * d + 1] = f.y;
      } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.kv) + at + 2 * d);
        k[2 * d] = bf16_lo(v), k[2 * d + 1] = bf16_hi(v);
      }
    }
    float sum = 0.f;
    for (int g = 0; g < p.rows; ++g) {
      if (p.causal && t >= n - p.s_q + g / p.H + 1) continue;
      const int64_t row = static_cast<int64_t>(b) * p.rows + g;
      const float lse = __ldg(p.lse + row);
      if (lse == -INFINITY) continue;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + row * kDimQK + lane * 18);
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < 9; ++d) {
        const uint32_t v = __ldg(q + d);
        s = fmaf(bf16_lo(v), k[2 * d], s);
        s = fmaf(bf16_hi(v), k[2 * d + 1], s);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      constexpr float kLog2e = 1.4426950408889634f;
      sum += fast_exp2(fmaf(s, p.scale_hi, fmaf(s, p.scale_lo, -lse * kLog2e)));
    }
    if (lane == 0) p.weights[b * p.weights_stride + t] += sum;
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status_t weights_impl(const mla_bf16_t* q, const float* lse, const void* kv_cache, bool fp8, float kv_scale,
                          int64_t num_blocks, const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B,
                          int s_q, int H, float softmax_scale, int causal_s_q, float* weights, int64_t weights_stride,
                          mla_stream_t stream) {
  if (!q || !lse || !kv_cache || !block_table || !seqlens || !weights) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || H < 1 || num_blocks < 1 || max_blocks < 1 || weights_stride < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(weights, 4))
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(s_q) * H > kRowsPerPair * kMaxPairsPerCluster || B > kScheduleMaxB) return MLA_ERR_UNSUPPORTED;
  if (num_blocks * kPageTokens > (int64_t(1) << 31) - kPageTokens) return MLA_ERR_UNSUPPORTED;
  WeightsParams p = {};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.lse = lse;
  p.kv = kv_cache;
  p.kv_scale = kv_scale;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.B = B;
  p.s_q = s_q;
  p.H = H;
  p.rows = s_q * H;
  p.causal = causal_s_q ? 1 : 0;
  int64_t slots = static_cast<int64_t>(max_blocks) * kPageTokens;
  slots = slots < weights_stride ? slots : weights_stride;
  p.slots = static_cast<int>(slots < INT32_MAX ? slots : INT32_MAX);
  const double scale = static_cast<double>(softmax_scale) * 1.4426950408889634074 * (fp8 ? kv_scale : 1.0);
  p.scale_hi = static_cast<float>(scale);
  p.scale_lo = static_cast<float>(scale - static_cast<double>(p.scale_hi));
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.status = device_status_word();
  if (!p.status) return MLA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(static_cast<unsigned>((p.slots + kPageTokens - 1) / kPageTokens), static_cast<unsigned>(B)), dim3(256),
                 0, reinterpret_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = fp8 ? cudaLaunchKernelEx(&cfg, mla_attn_weights_kernel<true>, p)
                            : cudaLaunchKernelEx(&cfg, mla_attn_weights_kernel<false>, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_attn_weights(const mla_bf16_t* q, const float* lse, const mla_bf16_t* kv_cache, int64_t num_blocks,
                              const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B, int s_q, int H,
                              float softmax_scale, int causal_s_q, float* weights, int64_t weights_stride,
                              mla_stream_t stream) {
  return weights_impl(q, lse, kv_cache, false, 1.f, num_blocks, block_table, max_blocks, seqlens, B, s_q, H,
                      softmax_scale, causal_s_q, weights, weights_stride, stream);
}

mla_status_t mla_attn_weights_fp8(const mla_bf16_t* q, const float* lse, const uint8_t* kv_cache, float kv_scale,
                                  int64_t num_blocks, const int32_t* block_table, int max_blocks,
                                  const int32_t* seqlens, int B, int s_q, int H, float softmax_scale, int causal_s_q,
                                  float* weights, int64_t weights_stride, mla_stream_t stream) {
  return weights_impl(q, lse, kv_cache, true, kv_scale, num_blocks, block_table, max_blocks, seqlens, B, s_q, H,
                      softmax_scale, causal_s_q, weights, weights_stride, stream);
}

}  // extern "C"
