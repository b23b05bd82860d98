// pda_cvt.cuh -- conversions between fp32 pairs and packed bf16 or E4M3, one
// instruction each. Internal to each translation unit.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pda {
namespace {

// Two floats -> two E4M3 codes (RNE, saturating to +-448): low byte from `lo`.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes -> two floats (exact): .x from the low byte.
__device__ __forceinline__ float2 e4m3x2_to_f2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Two floats -> two bf16 (RNE): low half from `lo`.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace
}  // namespace pda
