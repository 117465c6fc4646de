// Norm behind a block, its gate and scale, the residual, and the norm ahead of the
// next block with its MX codes, in one pass:
//   n = x / sqrt(mean(x^2) + eps) * w_post      (or x)
//   z = residual_scale * residual + block_scale * act(gate) * n,  residual_out = z
//   y = z / sqrt(mean(z^2) + eps) * w,  (codes, scales) = MX(y)
// One CTA holds one row in registers through both sums of squares, so every input is
// read once and every output written once; the residual and a gate of the row's own
// are on their way before the first sum is.  The bound is HBM for many rows and the
// latency of a launch, two block-wide sums and their loads for few.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace mxk {

namespace {

// Threads of a row: twice as many leave no room for another row's loads beside them, half as
// many hold twice as much of it (in us, by 256 / 512 / 1024, bf16 unless said: 32 x 4096 3.2 / 2.7 /
// 2.7, 32 x 16384 6.8 / 5.0 / 4.6, 8192 x 4096 56 / 56 / 56, in fp32 with a gate for each element
// 84 / 84 / 96, 8192 x 8192 98 / 114 / 163, 4096 x 16384 142 / 103 / 137, 2048 x 32768 243 / 150 / 114).
constexpr int kMostThreads = 512;

// Sum over the block, the same bits in every thread: warps add in a fixed order.
__device__ __forceinline__ float block_sum(float v, float* warp_sum) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (lane == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  float total = lane < static_cast<int>(blockDim.x >> 5) ? warp_sum[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  return total;
}

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// Eight elements of a vector that is the same for all rows (from L1 or L2 after the first).
__device__ __forceinline__ void load_vec8(const void* p, int64_t i, bool f32, float (&v)[8]) {
  if (f32) load8<true>(p, i, v);
  else load8<false>(p, i, v);
}

// sigmoid.  Where the residual is bf16, as all that is left are then bf16 or MX codes: by the
// quick exponential, whose error grows with |g| to 2^-17; beyond |g| = 87 the quotient's limits
// 0 and 1.  In fp32: 1 / (1 + e) or e / (1 + e) with e = exp(-|g|), which loses no small result,
// as 2^t with t = -|g| log2(e) in two floats: 2^-22 (2^t) + 2^-24 + 2^-24 (1 + e) + 2^-22 (the
// quick division, 2 ulp for divisors of this size) off for any g (8192 x 4096 with a gate for
// each element, L2 flushed: 94.9 us, by the quick one 92.8).
template <bool F32>
__device__ __forceinline__ float gate_of(float g, int act) {
  if (!act) return g;
  if (!F32) return __fdividef(1.0f, 1.0f + __expf(-g));
  const float a = -fabsf(g), t = a * 1.44269502f;                              // log2(e), and what its float leaves out
  const float rest = fmaf(a, 1.92596303e-8f, fmaf(a, 1.44269502f, -t));
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e, rest * 0.69314718f, e);
  return __fdividef(g < 0.0f ? e : 1.0f, 1.0f + e);
}

// NC groups of eight elements a thread; XF32, RF32: x, residual are fp32, else bf16;
// GATE: 0 none, one a channel or one a token, 1 [T, H] bf16, 2 [T, H] fp32.
// Rows of up to 16 elements a thread hold the residual and the gate beside x; longer ones
// have no registers for that and load them behind the first sum.
template <int NC, bool XF32, bool RF32, int GATE>
__global__ void __launch_bounds__(kMostThreads) k_sandwich_rmsnorm(const SandwichArgs a) {
  constexpr bool kEarly = NC <= 2;
  constexpr int NE = kEarly ? NC : 1;
  __shared__ float sums[2][32];
  const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
  const int n8 = a.H / 8;
  const int64_t t = blockIdx.x, row8 = t * n8;
  float z[NC][8], r[NE][8], g[NE][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * nt + tid;
#pragma unroll
    for (int m = 0; m < 8; ++m) z[c][m] = 0.0f;
    if (i < n8) {
      load8<XF32>(a.x, row8 + i, z[c]);
      if (kEarly) {
        load8<RF32>(a.residual, row8 + i, r[c % NE]);
        if (GATE) load8<GATE == 2>(a.gate, row8 + i, g[c % NE]);
      }
    }
  }
  const float token_gate = a.gate_kind == MX_GATE_TOKEN ? gate_of<RF32>(load1(a.gate, t, a.gate_f32), a.gate_act) : 1.0f;
  float inv = 1.0f;
  if (a.post_weight) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int m = 0; m < 8; ++m) ss = fmaf(z[c][m], z[c][m], ss);
    }
    inv = __frsqrt_rn(block_sum(ss, sums[0]) / static_cast<float>(a.H) + a.eps);
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * nt + tid;
    if (i < n8) {
      if (!kEarly) {
        load8<RF32>(a.residual, row8 + i, r[0]);
        if (GATE) load8<GATE == 2>(a.gate, row8 + i, g[0]);
      }
      if (a.post_weight) {
        float w[8];
        load_vec8(a.post_weight, i, a.post_weight_f32, w);
#pragma unroll
        for (int m = 0; m < 8; ++m) z[c][m] = z[c][m] * inv * w[m];
      }
      if (GATE) {
#pragma unroll
        for (int m = 0; m < 8; ++m) z[c][m] *= gate_of<RF32>(g[c % NE][m], a.gate_act);
      } else if (a.gate_kind == MX_GATE_CHANNEL) {
        float w[8];
        load_vec8(a.gate, i, a.gate_f32, w);
#pragma unroll
        for (int m = 0; m < 8; ++m) z[c][m] *= gate_of<RF32>(w[m], a.gate_act);
      } else if (a.gate_kind == MX_GATE_TOKEN) {
#pragma unroll
        for (int m = 0; m < 8; ++m) z[c][m] *= token_gate;
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        z[c][m] = fmaf(a.block_scale, z[c][m], a.residual_scale * r[c % NE][m]);
        ss = fmaf(z[c][m], z[c][m], ss);
      }
      if (RF32) {
        float4* o = static_cast<float4*>(a.residual_out) + 2 * (row8 + i);
        o[0] = make_float4(z[c][0], z[c][1], z[c][2], z[c][3]);
        o[1] = make_float4(z[c][4], z[c][5], z[c][6], z[c][7]);
      } else {
        static_cast<uint4*>(a.residual_out)[row8 + i] = pack_bf16x8(z[c]);
      }
    }
  }
  if (!a.weight) return;
  inv = __frsqrt_rn(block_sum(ss, sums[1]) / static_cast<float>(a.H) + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = c * nt + tid;
    const bool in = i < n8;  // the same for the four lanes of a block: H is a multiple of 32
    if (in) {
      float w[8];
      load_vec8(a.weight, i, a.weight_f32, w);
#pragma unroll
      for (int m = 0; m < 8; ++m) z[c][m] = z[c][m] * inv * w[m];
      if (a.y) static_cast<uint4*>(a.y)[row8 + i] = pack_bf16x8(z[c]);
    }
    if (a.codes) {
      uint8_t scale;
      const uint2 codes = mx_codes8(z[c], a.e2m1 != 0, scale);  // from the fp32 y: one rounding
      if (in) {
        if (a.e2m1) reinterpret_cast<uint32_t*>(a.codes)[row8 + i] = codes.x;
        else reinterpret_cast<uint2*>(a.codes)[row8 + i] = codes;
        if ((lane & 3) == 0) a.scales[(row8 + i) >> 2] = scale;
      }
    }
  }
}

template <int NC, bool XF32, bool RF32>
void launch_gate(const SandwichArgs& a, int threads, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.T);
  if (a.gate_kind != MX_GATE_FULL) k_sandwich_rmsnorm<NC, XF32, RF32, 0><<<grid, threads, 0, s>>>(a);
  else if (!a.gate_f32) k_sandwich_rmsnorm<NC, XF32, RF32, 1><<<grid, threads, 0, s>>>(a);
  else k_sandwich_rmsnorm<NC, XF32, RF32, 2><<<grid, threads, 0, s>>>(a);
}

template <int NC>
cudaError_t launch_nc(const SandwichArgs& a, int threads, cudaStream_t s) {
  if (a.x_f32) {
    if (a.residual_f32) launch_gate<NC, true, true>(a, threads, s);
    else launch_gate<NC, true, false>(a, threads, s);
  } else {
    if (a.residual_f32) launch_gate<NC, false, true>(a, threads, s);
    else launch_gate<NC, false, false>(a, threads, s);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sandwich_rmsnorm(const SandwichArgs& a, cudaStream_t s) {
  const int n8 = a.H / 8;
  int nc = 1;
  while (nc < 8 && (n8 + nc - 1) / nc > kMostThreads) nc *= 2;
  const int threads = ((n8 + nc - 1) / nc + 31) / 32 * 32;
  switch (nc) {
    case 1: return launch_nc<1>(a, threads, s);
    case 2: return launch_nc<2>(a, threads, s);
    case 4: return launch_nc<4>(a, threads, s);
    default: return launch_nc<8>(a, threads, s);
  }
}

}  // namespace mxk
