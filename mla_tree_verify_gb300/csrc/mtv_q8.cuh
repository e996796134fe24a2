// Shared by the kernels of the 8-bit latent cache: e4m3 conversions and the scale rule.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace mtv {
namespace q8 {

constexpr int kRow = 576;                 // bytes of a cache row: 512 latent, 64 rope dims
constexpr float kMax = 448.f;             // largest e4m3 value
constexpr uint32_t kNanCode4 = 0x7f7f7f7fu;
// Scales lie in [2^-40, 2^40].  The ratio of two of them, 2^80, leaves the softmax 46 binary
// orders before a weight of the smaller scale underflows fp32.
constexpr float kScaleMin = 0x1p-40f, kScaleMax = 0x1p40f;

__device__ __forceinline__ bool scale_ok(float s) { return s >= kScaleMin && s <= kScaleMax; }

// Two values to e4m3 (lo in the low byte), round to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  return pack2(a, b) | (pack2(c, d) << 16);
}
// Two e4m3 codes (low 16 bits) to f16x2: exact.
__device__ __forceinline__ uint32_t unpack2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  return r;
}

}  // namespace q8
}  // namespace mtv
