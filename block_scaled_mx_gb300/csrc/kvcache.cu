// The paged MX cache: quantising new keys and values as they are written, and
// reading them back as bf16.  Both are memory-bound; a warp takes one token (its
// page is looked up once) and each lane 16-byte groups of it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace mxk {

namespace {

constexpr int kWarps = 4;   // tokens of a block
constexpr int kUnroll = 4;  // groups of eight elements of K, and of V, that a lane loads before it uses one

// Cache row (page, place) of token t: the sequence that holds it by a 32-way
// search of q_starts, its position counted back from the sequence's length.
// Returns the row index (page * n_kv_heads) * page_size + place of head 0, or
// -1 for a token past the last sequence; bad metadata sets the status word.
__device__ __forceinline__ int64_t token_row(const KvArgs& a, int t, int lane) {
  int lo = 0, hi = a.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && a.q_starts[i] <= t;
    const int n = max(__popc(__ballot_sync(0xffffffffu, le)), 1);
    lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  const int start = a.q_starts[lo], end = a.q_starts[lo + 1], kv = a.kv_lens[lo];
  if (t >= end) return -1;
  const int64_t pos = static_cast<int64_t>(kv) - (end - t);
  if (start < 0 || start > t || end > a.T || pos < 0 || kv > static_cast<int64_t>(a.max_pages) * a.page_size) {
    if (lane == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
    return -1;
  }
  const int p = static_cast<int>(pos / a.page_size);
  const int page = a.block_table[static_cast<int64_t>(lo) * a.max_pages + p];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
    return -1;
  }
  return static_cast<int64_t>(page) * a.n_heads * a.page_size + (pos - static_cast<int64_t>(p) * a.page_size);
}

// Lane items are groups of eight elements of K, then of V; four consecutive
// lanes hold one MX block (head_dim is a multiple of 32, so blocks and heads
// start at multiples of four lanes).  All of a lane's loads are under way before
// the token's place is looked up, three dependent loads later; with K and V in
// one warp a look-up serves up to 4 KB (8932 tokens of 8 x 128: one tensor a warp
// 13.8 us, both 10.8; the bytes at copy rate take 8.2).
template <bool E2M1>
__global__ void __launch_bounds__(32 * kWarps) k_kv_append(const KvArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int per_head = a.head_dim / 8, n = a.n_heads * per_head;
  const uint4* k = static_cast<const uint4*>(a.k) + static_cast<int64_t>(t) * a.k_stride / 8;
  const uint4* v = static_cast<const uint4*>(a.v) + static_cast<int64_t>(t) * a.v_stride / 8;
  const int i0 = blockIdx.y * 32 * kUnroll + lane;
  uint4 w[2][kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = min(i0 + 32 * u, n - 1);
    w[0][u] = __ldg(k + i);
    w[1][u] = __ldg(v + i);
  }
  const int64_t row0 = token_row(a, t, lane);
  if (row0 < 0) return;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = i0 + 32 * u;
    if (i - lane >= n) break;
    const int h = i / per_head, e = i - h * per_head;
    const int64_t row = row0 + static_cast<int64_t>(h) * a.page_size;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t b[4] = {w[x][u].x, w[x][u].y, w[x][u].z, w[x][u].w};
      uint32_t amax = 0;
#pragma unroll
      for (int m = 0; m < 4; ++m) amax = max(amax, max(b[m] & 0x7FFFu, (b[m] >> 16) & 0x7FFFu));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int s = mx_block_exponent(amax << 16, E2M1 ? 2 : 8);
      const float p = pow2_neg(s);
      uint32_t c[2] = {0u, 0u};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float x0 = __uint_as_float(b[m] << 16) * p, x1 = __uint_as_float(b[m] & 0xFFFF0000u) * p;
        if (E2M1) c[0] |= (enc_e2m1(x0) | (enc_e2m1(x1) << 4)) << (8 * m);
        else c[m >> 1] |= enc_e4m3x2(x0, x1) << ((m & 1) * 16);
      }
      if (i < n) {
        uint8_t* codes = x ? a.v_codes : a.k_codes;
        if (E2M1) reinterpret_cast<uint32_t*>(codes)[row * per_head + e] = c[0];
        else reinterpret_cast<uint2*>(codes)[row * per_head + e] = make_uint2(c[0], c[1]);
        if ((lane & 3) == 0) (x ? a.v_scales : a.k_scales)[row * (per_head / 4) + e / 4] = static_cast<uint8_t>(s + 127);
      }
    }
  }
}

// The same lane items, the other way round.  The loads wait for the look-up here,
// so a lane has eight of them, and their scales, under way at once (one tensor a
// warp: 29.2 us for 26370 tokens of 8 x 128, both: 28.2; sixteen
// elements a lane wrote half sectors: 33.9).
template <bool E2M1>
__global__ void __launch_bounds__(32 * kWarps) k_kv_read(const KvArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int per_head = a.head_dim / 8, n = a.n_heads * per_head;
  const int i0 = blockIdx.y * 32 * kUnroll + lane;
  const int64_t row0 = token_row(a, t, lane);
  uint2 c[2][kUnroll];
  int s[2][kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = min(i0 + 32 * u, n - 1), h = i / per_head, e = i - h * per_head;
    const int64_t row = max(row0, static_cast<int64_t>(0)) + static_cast<int64_t>(h) * a.page_size;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* codes = x ? a.v_codes : a.k_codes;
      if (E2M1) c[x][u] = make_uint2(reinterpret_cast<const uint32_t*>(codes)[row * per_head + e], 0u);
      else c[x][u] = reinterpret_cast<const uint2*>(codes)[row * per_head + e];
      s[x][u] = (x ? a.v_scales : a.k_scales)[row * (per_head / 4) + e / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = i0 + 32 * u;
    if (i >= n) break;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float p = e8m0_value(s[x][u]);
      uint32_t o[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t h2;
        if (E2M1) h2 = f16x2_of_e2m1x2((c[x][u].x >> (8 * m)) & 0xFFu);
        else h2 = f16x2_of_e4m3x2(((m < 2 ? c[x][u].x : c[x][u].y) >> (16 * (m % 2))) & 0xFFFFu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * p, f.y * p);
        o[m] = row0 < 0 ? 0u : *reinterpret_cast<const uint32_t*>(&b);
      }
      // evict-first: what was written pushes no cache row out (28.2 -> 26.8 us in the case above)
      __stcs(static_cast<uint4*>(x ? a.v_out : a.k_out) + static_cast<int64_t>(t) * n + i, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

dim3 kv_grid(const KvArgs& a) {
  const int n = a.n_heads * a.head_dim / 8;
  return dim3(static_cast<unsigned>((a.T + kWarps - 1) / kWarps), static_cast<unsigned>((n + 32 * kUnroll - 1) / (32 * kUnroll)));
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, cudaStream_t s) {
  if (a.e2m1) k_kv_append<true><<<kv_grid(a), 32 * kWarps, 0, s>>>(a);
  else k_kv_append<false><<<kv_grid(a), 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvArgs& a, cudaStream_t s) {
  if (a.e2m1) k_kv_read<true><<<kv_grid(a), 32 * kWarps, 0, s>>>(a);
  else k_kv_read<false><<<kv_grid(a), 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mxk
