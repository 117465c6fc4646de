// Residual addition, root-mean-square norm and MX quantisation in one pass:
//   z = x + residual,  residual_out = z,  y = z / sqrt(mean(z^2) + eps) * weight,
//   (codes, scales) = MX(y)
// One CTA holds one row of z in registers between the sum of squares and the
// scaling, so every input is read once and every output written once; the
// bound is HBM for many rows and launch latency for few.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace mxk {

namespace {

// NC groups of eight elements a thread; XF32: x is fp32, else bf16; RES: 0 no
// residual, 1 bf16, 2 fp32.  Four consecutive lanes hold one MX block of 32.
template <int NC, bool XF32, int RES>
__global__ void __launch_bounds__(1024) k_add_rmsnorm(const NormArgs a) {
  __shared__ float warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
  const int n8 = a.H / 8;
  const int64_t row8 = static_cast<int64_t>(blockIdx.x) * n8;
  float z[NC][8];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * nt + tid;
    if (i < n8) {
      load8<XF32>(a.x, row8 + i, z[c]);
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) z[c][m] = 0.0f;
    }
  }
  if (RES != 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * nt + tid;
      if (i < n8) {
        float r[8];
        load8<RES == 2>(a.residual, row8 + i, r);
#pragma unroll
        for (int m = 0; m < 8; ++m) z[c][m] += r[m];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int m = 0; m < 8; ++m) ss = fmaf(z[c][m], z[c][m], ss);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (lane == 0) warp_sum[tid >> 5] = ss;
  if (RES != 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * nt + tid;
      if (i < n8) {
        if (RES == 1) {
          static_cast<uint4*>(a.residual_out)[row8 + i] = pack_bf16x8(z[c]);
        } else {
          float4* o = static_cast<float4*>(a.residual_out) + 2 * (row8 + i);
          o[0] = make_float4(z[c][0], z[c][1], z[c][2], z[c][3]);
          o[1] = make_float4(z[c][4], z[c][5], z[c][6], z[c][7]);
        }
      }
    }
  }
  __syncthreads();
  // every warp adds the warps' sums in the same order
  float total = lane < (nt >> 5) ? warp_sum[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  const float inv = __frsqrt_rn(total / static_cast<float>(a.H) + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * nt + tid;
    const bool in = i < n8;  // the same for the four lanes of a block: H is a multiple of 32
    float w[8];
    if (in) {
      if (a.weight_f32) load8<true>(a.weight, i, w);
      else load8<false>(a.weight, i, w);
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) w[m] = 0.0f;
    }
    uint32_t amax = 0;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      z[c][m] = z[c][m] * inv * w[m];
      amax = max(amax, __float_as_uint(z[c][m]) & 0x7FFFFFFFu);
    }
    if (in && a.y) static_cast<uint4*>(a.y)[row8 + i] = pack_bf16x8(z[c]);
    if (a.codes) {
      // y goes to the codes from its fp32 value: one rounding, not two
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int s = mx_block_exponent(amax, a.e2m1 ? 2 : 8);
      const float p = pow2_neg(s);
      if (a.e2m1) {
        uint32_t packed = 0;
#pragma unroll
        for (int m = 0; m < 8; ++m) packed |= enc_e2m1(z[c][m] * p) << (4 * m);
        if (in) reinterpret_cast<uint32_t*>(a.codes)[row8 + i] = packed;
      } else {
        uint2 packed;
        packed.x = enc_e4m3x2(z[c][0] * p, z[c][1] * p) | (enc_e4m3x2(z[c][2] * p, z[c][3] * p) << 16);
        packed.y = enc_e4m3x2(z[c][4] * p, z[c][5] * p) | (enc_e4m3x2(z[c][6] * p, z[c][7] * p) << 16);
        if (in) reinterpret_cast<uint2*>(a.codes)[row8 + i] = packed;
      }
      if (in && (lane & 3) == 0) a.scales[(row8 + i) >> 2] = static_cast<uint8_t>(s + 127);
    }
  }
}

template <int NC>
cudaError_t launch_nc(const NormArgs& a, int threads, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.T);
  const int res = !a.residual ? 0 : a.residual_f32 ? 2 : 1;
  if (a.x_f32) {
    if (res == 0) k_add_rmsnorm<NC, true, 0><<<grid, threads, 0, s>>>(a);
    else if (res == 1) k_add_rmsnorm<NC, true, 1><<<grid, threads, 0, s>>>(a);
    else k_add_rmsnorm<NC, true, 2><<<grid, threads, 0, s>>>(a);
  } else {
    if (res == 0) k_add_rmsnorm<NC, false, 0><<<grid, threads, 0, s>>>(a);
    else if (res == 1) k_add_rmsnorm<NC, false, 1><<<grid, threads, 0, s>>>(a);
    else k_add_rmsnorm<NC, false, 2><<<grid, threads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

// Threads of a row up to which each takes one group of eight.  8192 rows of 4096
// bf16: 53.7 us with at most 128 threads, 51.0 with 256, 47.2 with 512 (the bytes
// at copy rate: 44.7); 2048 rows of 16384: 57.9 with 512, 67.9 with 1024, whose
// block leaves no room for another row's loads while it waits for its sum.
constexpr int kMostThreads = 512;

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  const int n8 = a.H / 8;
  int nc = 1;
  while (nc < 4 && (n8 + nc - 1) / nc > kMostThreads) nc *= 2;
  const int threads = ((n8 + nc - 1) / nc + 31) / 32 * 32;
  switch (nc) {
    case 1: return launch_nc<1>(a, threads, s);
    case 2: return launch_nc<2>(a, threads, s);
    default: return launch_nc<4>(a, threads, s);
  }
}

}  // namespace mxk
