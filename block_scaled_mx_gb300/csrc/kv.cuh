// Reading MX cache elements: E4M3 and E2M1 pairs to f16 (both are exact there)
// and E8M0 scales.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace mxk {

// Two E4M3 codes (low byte first) as f16x2.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Two E2M1 codes (one byte, low nibble first) as f16x2.
__device__ __forceinline__ uint32_t f16x2_of_e2m1x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "mov.b16 {b0, b1}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// 2^(code - 127) as fp32 (code 0 is the subnormal 2^-127, 255 is NaN).
__device__ __forceinline__ float e8m0_value(int code) {
  return __uint_as_float(code > 0 && code < 255 ? static_cast<uint32_t>(code) << 23 : code == 0 ? 1u << 22 : 0x7FC00000u);
}

}  // namespace mxk
