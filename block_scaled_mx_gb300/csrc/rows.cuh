// Rows of bf16 or fp32 in groups of eight elements (16 or 32 bytes a lane), and
// their MX codes where four consecutive lanes hold one block of 32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"

namespace mxk {

// Eight consecutive elements as fp32; `i` counts groups of eight.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if (F32) {
    const float4* q = static_cast<const float4*>(p) + 2 * i;
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = static_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v[2 * m] = __uint_as_float(w[m] << 16);
      v[2 * m + 1] = __uint_as_float(w[m] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * m], v[2 * m + 1]);
    w[m] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// E2M1 codes of two block-scaled values with the hardware conversion (round to nearest
// even, saturate at 6, keep the sign): `lo` in bits 0..3, `hi` in bits 4..7.
__device__ __forceinline__ uint32_t enc_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// MX codes of eight consecutive values of a lane, four lanes to a block of 32: the E4M3
// codes in .x and .y, or the E2M1 codes in .x.  Every lane of the warp calls it.
// `scale` gets the block's scale byte.
__device__ __forceinline__ uint2 mx_codes8(const float (&v)[8], bool e2m1, uint8_t& scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int m = 0; m < 8; ++m) amax = max(amax, __float_as_uint(v[m]) & 0x7FFFFFFFu);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int s = mx_block_exponent(amax, e2m1 ? 2 : 8);
  const float p = pow2_neg(s);
  scale = static_cast<uint8_t>(s + 127);
  uint2 c = make_uint2(0u, 0u);
  if (e2m1) {
#pragma unroll
    for (int m = 0; m < 4; ++m) c.x |= enc_e2m1x2(v[2 * m] * p, v[2 * m + 1] * p) << (8 * m);
  } else {
    c.x = enc_e4m3x2(v[0] * p, v[1] * p) | (enc_e4m3x2(v[2] * p, v[3] * p) << 16);
    c.y = enc_e4m3x2(v[4] * p, v[5] * p) | (enc_e4m3x2(v[6] * p, v[7] * p) << 16);
  }
  return c;
}

}  // namespace mxk
