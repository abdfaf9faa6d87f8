// The 4-bit latent cache: the layout of a cached row and the conversions of its codes.
//
// A row is 352 bytes (22 units of 16):
//   [0, 256)    512 E2M1 codes of the latent, dim 2i in the low half of byte i
//   [256, 288)  32 E4M3 scales, one for 16 latent dims
//   [288, 352)  64 E4M3 codes of the RoPE key
// latent value = code * scale * kv_scale, RoPE value = code * kv_scale.  A code has 2 significant bits and a scale 4,
// so code * scale is exact in fp16 (and at most 6 * 448); kv_scale is left to the scores and the output.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace mla {

constexpr int kFp4RowBytes = 352;
constexpr int kFp4Scales = 256, kFp4Rope = 288;   // byte offsets in a row
constexpr int kFp4Group = 16;                     // latent dims of a scale

// Scales for which the largest cached value, 6 * 448 * kv_scale, and the smallest step, 2^-10 kv_scale, are normal floats.
inline bool fp4_scale_ok(float kv_scale) { return kv_scale >= 0x1p-116f && kv_scale <= 0x1p115f; }

// Two floats as a pair of E2M1 codes (to nearest even, saturating at +-6): `lo` in bits 0..3, `hi` in 4..7.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The values of the pairs of E2M1 codes in byte b of w, as fp16 (low half: the byte's low code); exact.
template <int b>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t d;
  if constexpr (b == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (b == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (b == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
// The values of the two E4M3 codes in the low (half = 0) or high half of w, as fp16; exact.
template <int half>
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t d;
  if constexpr (half == 0)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The larger one, NaN if either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

}  // namespace mla
