// Absorbed MLA decode over the 4-bit latent cache (mla_fp4.cuh): dense and over lists of tokens.
// C entries at the end (declared in mla.h).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "mla_fp4.cuh"
#include "mla_kernels.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

constexpr int kTile = 32, kRowsCta = 8, kStride = kDimQK + 1;
constexpr size_t kSmem = sizeof(float) * (kTile * kStride + kRowsCta * kDimQK + kRowsCta * kTile + kRowsCta);

// A CTA takes eight query rows of a request past its tokens, 32 at a time, values as fp32 in shared memory.
__global__ void __launch_bounds__(256) mla_decode_fp4_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ float sm[];
  float* k = sm;
  float* q = k + kTile * kStride;
  float* pr = q + kRowsCta * kDimQK;
  float* alpha = pr + kRowsCta * kTile;
  griddep_wait();
  const int b = blockIdx.y, g0 = blockIdx.x * kRowsCta, tid = threadIdx.x, row = tid >> 5, lane = tid & 31;
  const int g = g0 + row;
  for (int i = tid; i < kRowsCta * kDimQK; i += 256) {
    const int r = g0 + i / kDimQK;
    q[i] = r < p.rows ? __bfloat162float(p.q[(static_cast<int64_t>(b) * p.rows + r) * kDimQK + i % kDimQK]) : 0.f;
  }
  const int n = p.lens[b], len = p.seqlens[b];
  const int last = p.causal ? len - p.s_q + (g < p.rows ? g / p.H : 0) : len - 1;   // the row sees positions up to here
  float acc[kRowsCta][2] = {};
  float m = -INFINITY, l = 0.f;
  for (int t0 = 0; t0 < n; t0 += kTile) {
    __syncthreads();
    for (int j = row; j < kTile; j += 8) {   // a warp a token
      const int e = t0 + j;
      int64_t at = -1;
      if (e < n) {
        int t = e;
        if (p.indices) t = e < p.idx_stride ? p.indices[b * p.idx_stride + e] : -1;
        if (t >= 0 && t < len && t / kPageTokens < p.max_blocks) {
          const int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + t / kPageTokens];
          if (blk >= 0 && blk < p.num_blocks) at = static_cast<int64_t>(blk) * kPageTokens + t % kPageTokens;
        }
        if (at < 0 && lane == 0) atomicCAS(p.status, 0, MLA_ERR_DEVICE_BOUNDS);
      }
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.kv) + at * kFp4RowBytes;
      float* dst = k + j * kStride;
      for (int i = lane; i < kDimQK; i += 32) {
        float v = 0.f;
        if (at >= 0 && i < kDimV) {
          const uint32_t pair = e2m1x2_to_f16x2<0>(src[i / 2]);
          const __half2 h = *reinterpret_cast<const __half2*>(&pair);
          v = (i & 1 ? __high2float(h) : __low2float(h)) * e4m3x2_to_float2(src[kFp4Scales + i / kFp4Group]).x;
        } else if (at >= 0) {
          v = e4m3x2_to_float2(src[kFp4Rope + i - kDimV]).x;
        }
        dst[i] = v;
      }
    }
    __syncthreads();
    {
      const int e = t0 + lane;
      float s = -INFINITY;
      int t = e;
      if (p.indices && e < n) t = e < p.idx_stride ? p.indices[b * p.idx_stride + e] : -1;
      if (e < n && g < p.rows && t <= last) {
        s = 0.f;
        for (int i = 0; i < kDimQK; ++i) s = fmaf(q[row * kDimQK + i], k[lane * kStride + i], s);
        s *= p.scale_log2 * p.kv_scale;
      }
      float mx = s;
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;
      const float e2 = exp2f(s - ref);
      float sum = e2;
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float a = exp2f(m - ref);
      l = l * a + sum;
      m = m_new;
      pr[row * kTile + lane] = e2;
      if (lane == 0) alpha[row] = a;
    }
    __syncthreads();
    for (int r = 0; r < kRowsCta; ++r) acc[r][0] *= alpha[r], acc[r][1] *= alpha[r];
    for (int j = 0; j < min(kTile, n - t0); ++j) {
      const float v0 = k[j * kStride + 2 * tid], v1 = k[j * kStride + 2 * tid + 1];
      for (int r = 0; r < kRowsCta; ++r) acc[r][0] += pr[r * kTile + j] * v0, acc[r][1] += pr[r * kTile + j] * v1;
    }
  }
  __syncthreads();
  if (lane == 0) {
    alpha[row] = l == 0.f ? 0.f : p.kv_scale / l;
    if (g < p.rows) p.lse[static_cast<int64_t>(b) * p.rows + g] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
  __syncthreads();
  for (int r = 0; r < kRowsCta && g0 + r < p.rows; ++r)
    reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(b) * p.rows + g0 + r) * kDimV)[tid] =
        pack_bf16x2(acc[r][0] * alpha[r], acc[r][1] * alpha[r]);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mla_status_t decode_fp4_impl(const void* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                             const int32_t* block_table, int max_blocks, const int32_t* seqlens, const int32_t* indices,
                             int64_t index_stride, const int32_t* topk_lens, int B, int s_q, int H, float softmax_scale,
                             int causal_s_q, const void* metadata, int num_sm_parts, void* workspace,
                             size_t workspace_bytes, mla_bf16_t* out, float* lse, mla_stream_t stream) {
  if (!q || !kv_cache || !block_table || !seqlens || !metadata || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || H < 1 || num_blocks < 1 || max_blocks < 1 || num_sm_parts < 1) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(metadata, 4))
    return MLA_ERR_INVALID_ARG;
  if (indices && (!topk_lens || index_stride < 1 || !aligned(indices, 4) || !aligned(topk_lens, 4))) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(kv_scale) || !(kv_scale > 0.f) || !fp4_scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  const double scale_log2 = static_cast<double>(softmax_scale) * 1.4426950408889634074;
  if (!std::isnormal(static_cast<float>(scale_log2 * kv_scale))) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(s_q) * H > kMaxPairsPerCluster * kRowsPerPair || B > kScheduleMaxB) return MLA_ERR_UNSUPPORTED;
  if (num_blocks > ((int64_t(1) << 31) - kPageTokens) / kPageTokens) return MLA_ERR_UNSUPPORTED;
  const int rows = s_q * H;
  const size_t need = mla_decode_workspace_size(B, s_q, H, num_sm_parts);
  if (workspace_bytes < need || !workspace) return MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  DecodeParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kv = reinterpret_cast<const __nv_bfloat16*>(kv_cache);
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.seqlens = seqlens;
  p.lens = indices ? topk_lens : seqlens;
  p.indices = indices;
  p.idx_stride = indices ? index_stride : 0;
  p.B = B;
  p.s_q = s_q;
  p.H = H;
  p.rows = rows;
  p.n_rb = (rows + kRowsPerPair - 1) / kRowsPerPair;
  p.scale_log2 = static_cast<float>(scale_log2);
  p.causal = causal_s_q ? 1 : 0;
  p.kv_scale = kv_scale;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = device_status_word();
  if (!p.status) return MLA_ERR_CUDA;
  if (cudaFuncSetAttribute(mla_decode_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(static_cast<unsigned>((rows + kRowsCta - 1) / kRowsCta), static_cast<unsigned>(B)), dim3(256), kSmem,
                 reinterpret_cast<cudaStream_t>(stream), attr);
  return cudaLaunchKernelEx(&cfg, mla_decode_fp4_kernel, p) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_decode_fp4(const mla_bf16_t* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                            const int32_t* block_table, int max_blocks, const int32_t* seqlens, int B, int s_q, int H,
                            float softmax_scale, int causal_s_q, const void* metadata, int num_sm_parts,
                            void* workspace, size_t workspace_bytes, mla_bf16_t* out, float* lse, mla_stream_t stream) {
  return decode_fp4_impl(q, kv_cache, kv_scale, num_blocks, block_table, max_blocks, seqlens, nullptr, 0, nullptr, B, s_q, H,
                         softmax_scale, causal_s_q, metadata, num_sm_parts, workspace, workspace_bytes, out, lse, stream);
}

mla_status_t mla_decode_sparse_fp4(const mla_bf16_t* q, const uint8_t* kv_cache, float kv_scale, int64_t num_blocks,
                                   const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                   const int32_t* indices, int64_t index_stride, const int32_t* topk_lens, int B, int s_q,
                                   int H, float softmax_scale, int causal_s_q, const void* metadata, int num_sm_parts,
                                   void* workspace, size_t workspace_bytes, mla_bf16_t* out, float* lse,
                                   mla_stream_t stream) {
  if (!indices) return MLA_ERR_INVALID_ARG;
  return decode_fp4_impl(q, kv_cache, kv_scale, num_blocks, block_table, max_blocks, seqlens, indices, index_stride,
                         topk_lens, B, s_q, H, softmax_scale, causal_s_q, metadata, num_sm_parts, workspace,
                         workspace_bytes, out, lse, stream);
}

}  // extern "C"
