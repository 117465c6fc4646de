// Rotary positions on the way into the paged MX cache: queries are rotated to bf16,
// keys rotated and quantised into their page, values quantised into theirs.
//
// A pair (a, b) of a head's first R elements at position p becomes
//   (a cos - b sin, a sin + b cos) * amplitude,  angle = p * f_i
// for the pairs (i, i + R/2) or (2i, 2i + 1).  Angles of far positions lose their
// fraction of a turn in fp32, so f_i is kept as the 64-bit fraction of a turn a
// position, p * f_i is a product modulo 2^64, which is exact but for f_i's own rounding
// (2^-52 turns a position), and its upper 32 bits are the angle in [-1/2, 1/2) turns (2^-32
// of a turn off).  Sines and products are fp32, a few 2^-24 of |a| + |b| off, where bf16 rounds
// by 2^-8 and E4M3 by 2^-4 of the result: of 67 million E4M3 codes of keys 97 are not those of
// 64-bit arithmetic (105 where sines are rounded from 64 bits, but each product to fp32).
//
// Memory-bound: every input is read once and every output written once.  A warp takes a
// token, or a part of one: its lanes find the angles' sines, each once, and go through the
// heads, a few at a time.  A lane holds eight elements of a head, so that four lanes are an
// MX block and the rotation's partner is a shuffle away (or in the lane itself), and the
// same eight of every head, so that its sines stay in registers.
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "rows.cuh"

namespace mxk {

namespace {

constexpr int kWarps = 4;        // of a block
constexpr int kUnroll = 4;       // groups of heads whose loads are under way together
constexpr int kMostPairs = 128;

enum Kind { kQuery, kKey, kValue };

// HALF: the pairs are (i, i + R/2).  `parts` warps share a token.
template <bool E2M1, bool HALF>
__global__ void __launch_bounds__(32 * kWarps) k_rope_kv_append(const RopeArgs r, int parts) {
  __shared__ __align__(16) float2 turned_of[kWarps][kMostPairs];  // (cos, sin) of the warp's token's pairs, times the amplitude
  const KvArgs& a = r.kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(w / parts), part = static_cast<int>(w - static_cast<int64_t>(t) * parts);
  if (t >= a.T) return;
  const int per_head = a.head_dim / 8, together = 32 / per_head, wide = together * per_head;  // heads and groups of eight of a warp's load
  const int hl = lane / per_head, e = lane - hl * per_head;                                   // which head, and group in it
  const int nq = (r.n_q_heads + together - 1) / together, nk = (a.n_heads + together - 1) / together;
  const int units = nq + 2 * nk;  // queries, then keys, then values
  const int u0 = units * part / parts, u1 = units * (part + 1) / parts;

  int64_t pos = 0;
  const int64_t row0 = token_row(a, t, lane, pos);
  if (row0 < 0) return;
  if (r.positions) pos = r.positions[t];

  const int half = r.rot / 16;  // groups of eight of half of the rotated part
  const bool turns = 8 * e < r.rot && hl < together;
  const bool second = HALF && e >= half;  // of the pairs: the sine has the other sign
  const int partner = second ? lane - half : lane + half;
  constexpr int kAngles = HALF ? 8 : 4;
  float cs[kAngles], sn[kAngles];
  if (u0 < nq + nk) {
    float2* const turned = turned_of[warp];
    for (int i = lane; i < r.rot / 2; i += 32) {
      const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(r.turns + i);
      // half turns, in [-1, 1): the product's upper word, its first 24 bits as a float and
      // the others by the derivative
      const uint32_t word = static_cast<uint32_t>(turn >> 32);
      const float h = static_cast<float>(static_cast<int32_t>(word & 0xFFFFFF00u));
      const float left = static_cast<float>(word & 0xFFu) * (3.14159274f * 0x1p-31f);
      float sine, cosine;
      sincospif(h * 0x1p-31f, &sine, &cosine);
      turned[i] = make_float2(fmaf(-sine, left, cosine) * r.amplitude, fmaf(cosine, left, sine) * r.amplitude);
    }
    __syncwarp();
    const float4* const mine = reinterpret_cast<const float4*>(turned + (turns ? HALF ? 8 * (second ? e - half : e) : 4 * e : 0));
#pragma unroll
    for (int i = 0; i < kAngles; i += 2) {
      const float4 c = mine[i / 2];
      cs[i] = c.x;
      sn[i] = second ? -c.y : c.y;
      cs[i + 1] = c.z;
      sn[i + 1] = second ? -c.w : c.w;
    }
  }

  // units [from, to) of one kind: a token's row of groups of eight, `wide` a unit
  auto go = [&](const uint4* src, int heads, int from, int to, auto kind_of) {
    constexpr Kind kKind = decltype(kind_of)::value;
    const int n = heads * per_head;
    for (int u = from; u < to; u += kUnroll) {
      uint4 x[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int g = (u + i) * wide + lane;
        x[i] = u + i < to && lane < wide && g < n ? __ldcs(src + g) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        if (u + i >= to) break;
        const int g = (u + i) * wide + lane;
        const bool in = lane < wide && g < n;
        const uint32_t b[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float o[8];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          o[2 * m] = __uint_as_float(b[m] << 16);
          o[2 * m + 1] = __uint_as_float(b[m] & 0xFFFF0000u);
        }
        if (kKind != kValue) {
          if (HALF) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t p = __shfl_sync(0xffffffffu, b[m], partner);
              if (turns) {
                o[2 * m] = fmaf(o[2 * m], cs[(2 * m) % kAngles], -__uint_as_float(p << 16) * sn[(2 * m) % kAngles]);
                o[2 * m + 1] = fmaf(o[2 * m + 1], cs[(2 * m + 1) % kAngles], -__uint_as_float(p & 0xFFFF0000u) * sn[(2 * m + 1) % kAngles]);
              }
            }
          } else if (turns) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float c = o[2 * m], d = o[2 * m + 1];
              o[2 * m] = fmaf(c, cs[m], -d * sn[m]);
              o[2 * m + 1] = fmaf(c, sn[m], d * cs[m]);
            }
          }
        }
        if (kKind == kQuery) {
          if (in) __stcs(static_cast<uint4*>(r.q_out) + static_cast<int64_t>(t) * r.q_out_stride / 8 + g, pack_bf16x8(o));
        } else {
          uint8_t scale;
          const uint2 c = mx_codes8(o, E2M1, scale);  // from the rotated fp32 values: one rounding
          if (in) {
            const int h = (u + i) * together + hl;
            const int64_t at = (row0 + static_cast<int64_t>(h) * a.page_size) * per_head + e;
            uint8_t* const codes = kKind == kKey ? a.k_codes : a.v_codes;
            if (E2M1) reinterpret_cast<uint32_t*>(codes)[at] = c.x;
            else reinterpret_cast<uint2*>(codes)[at] = c;
            if ((lane & 3) == 0) (kKind == kKey ? a.k_scales : a.v_scales)[at / 4] = scale;
          }
        }
      }
    }
  };
  const int k0 = nq, v0 = nq + nk;
  go(static_cast<const uint4*>(r.q) + static_cast<int64_t>(t) * r.q_stride / 8, r.n_q_heads, u0, min(u1, k0), std::integral_constant<Kind, kQuery>());
  go(static_cast<const uint4*>(a.k) + static_cast<int64_t>(t) * a.k_stride / 8, a.n_heads, max(u0, k0) - k0, min(u1, v0) - k0,
     std::integral_constant<Kind, kKey>());
  go(static_cast<const uint4*>(a.v) + static_cast<int64_t>(t) * a.v_stride / 8, a.n_heads, max(u0, v0) - v0, u1 - v0, std::integral_constant<Kind, kValue>());
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeArgs& r, cudaStream_t s) {
  const int together = 32 / (r.kv.head_dim / 8);
  const int units = (r.n_q_heads + together - 1) / together + 2 * ((r.kv.n_heads + together - 1) / together);
  // warps that share a token: as many as its groups of heads allow while the tokens alone
  // leave SMs idle (in us, 32 + 2 x 8 heads of 128, by 1 / 2 / 4 / 8 warps: one token 6.2 / 4.7 /
  // 4.1 / 3.7, 128 tokens 7.5 / 5.6 / 4.7 / 4.5, 600 tokens 6.8 / 5.7 / 5.6 / 7.3, 2048 tokens
  // 10.5 / 10.0 / 12.4 / 16.4, 8192 tokens 33.2 / 34.5 / 41.8 / 58.4)
  int parts = 1;
  while (parts < 16 && 2 * parts * 3 <= units + 3 && static_cast<int64_t>(r.kv.T) * parts < 152 * 16) parts *= 2;
  const int64_t warps = static_cast<int64_t>(r.kv.T) * parts;
  const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
  if (r.kv.e2m1) {
    if (r.interleaved) k_rope_kv_append<true, false><<<grid, 32 * kWarps, 0, s>>>(r, parts);
    else k_rope_kv_append<true, true><<<grid, 32 * kWarps, 0, s>>>(r, parts);
  } else {
    if (r.interleaved) k_rope_kv_append<false, false><<<grid, 32 * kWarps, 0, s>>>(r, parts);
    else k_rope_kv_append<false, true><<<grid, 32 * kWarps, 0, s>>>(r, parts);
  }
  return cudaGetLastError();
}

}  // namespace mxk
