// Rotary positions on the way into the paged MX cache: queries are rotated to bf16,
// keys rotated and quantised into their page, values quantised into theirs.
//
// A pair (a, b) of a head's first R elements at position p becomes
//   (a cos - b sin, a sin + b cos) * amplitude,  angle = p * f_i
// for the pairs (i, i + R/2) or (2i, 2i + 1).  Angles of far positions lose their
// fraction of a turn in fp32, so f_i is kept as the 64-bit fraction of a turn a
// position, p * f_i is a product modulo 2^64, which is exact but for f_i's own rounding
// (2^-53), and its upper 32 bits are the angle in [-1/2, 1/2) turns (2^-33 of a turn off).
//
// Memory-bound: every input is read once and every output written once.  A warp
// takes one token, or a part of one; a lane holds eight elements of a head, so that
// four lanes are an MX block and the rotation's partner is a shuffle away (or in the
// lane itself), and has the same place in every head: the angles are found once a warp.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "rows.cuh"

namespace mxk {

namespace {

constexpr int kWarps = 4;   // of a block
constexpr int kUnroll = 4;  // groups of heads whose loads are under way together

// HALF: the pairs are (i, i + R/2).  `parts` warps share a token.
template <bool E2M1, bool HALF>
__global__ void __launch_bounds__(32 * kWarps) k_rope_kv_append(const RopeArgs r, int parts) {
  const KvArgs& a = r.kv;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / parts), part = static_cast<int>(w - static_cast<int64_t>(t) * parts);
  if (t >= a.T) return;
  const int per_head = a.head_dim / 8, together = 32 / per_head;  // heads of a warp's load
  const int hl = lane / per_head, e = lane - hl * per_head;       // which of them, group of eight in it
  const int nq = (r.n_q_heads + together - 1) / together, nk = (a.n_heads + together - 1) / together;
  const int units = nq + 2 * nk;                                  // queries, then keys, then values
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * part / parts);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / parts);
  const uint4* const q = static_cast<const uint4*>(r.q) + static_cast<int64_t>(t) * r.q_stride / 8;
  const uint4* const k = static_cast<const uint4*>(a.k) + static_cast<int64_t>(t) * a.k_stride / 8;
  const uint4* const v = static_cast<const uint4*>(a.v) + static_cast<int64_t>(t) * a.v_stride / 8;
  auto load = [&](int u) {
    const uint4* p = u < nq ? q : u < nq + nk ? k : v;
    const int h = (u < nq ? u : u < nq + nk ? u - nq : u - nq - nk) * together + hl;
    const bool in = u < u1 && hl < together && h < (u < nq ? r.n_q_heads : a.n_heads);
    return in ? __ldcs(p + static_cast<int64_t>(h) * per_head + e) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 x[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) x[i] = load(u0 + i);

  int64_t pos = 0;
  const int64_t row0 = token_row(a, t, lane, pos);
  if (row0 < 0) return;
  if (r.positions) pos = r.positions[t];

  // cos and sin of the lane's eight elements (HALF) or four pairs; half of the pairs'
  // second members take the sine with the other sign
  const int half = r.rot / 16;  // groups of eight of half of the rotated part
  const bool turns = 8 * e < r.rot && hl < together;
  const bool second = HALF && e >= half;
  constexpr int kAngles = HALF ? 8 : 4;
  float cs[kAngles], sn[kAngles];
  if (u0 < nq + nk) {
    const int i0 = HALF ? 8 * (second ? e - half : e) : 4 * e;
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
      if (turns) {
        const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(r.turns + i0 + i);
        // half turns, in [-1, 1): the product's upper word, its first 24 bits as a float and
        // the others by the derivative
        const uint32_t word = static_cast<uint32_t>(turn >> 32);
        const float h = static_cast<float>(static_cast<int32_t>(word & 0xFFFFFF00u));
        const float left = static_cast<float>(word & 0xFFu) * (3.14159274f * 0x1p-31f);
        float sine, cosine;
        sincospif(h * 0x1p-31f, &sine, &cosine);
        cs[i] = fmaf(-sine, left, cosine) * r.amplitude;
        sn[i] = fmaf(cosine, left, sine) * (second ? -r.amplitude : r.amplitude);
      }
    }
  }
  const int partner = second ? lane - half : lane + half;

  for (int ub = u0; ub < u1; ub += kUnroll) {
    uint4 next[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) next[i] = load(ub + kUnroll + i);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int u = ub + i;
      if (u >= u1) break;
      const int kind = u < nq ? 0 : u < nq + nk ? 1 : 2;
      const int h = (kind == 0 ? u : kind == 1 ? u - nq : u - nq - nk) * together + hl;
      const bool in = hl < together && h < (kind == 0 ? r.n_q_heads : a.n_heads);
      const uint32_t b[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float o[8];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        o[2 * m] = __uint_as_float(b[m] << 16);
        o[2 * m + 1] = __uint_as_float(b[m] & 0xFFFF0000u);
      }
      if (kind != 2) {
        if (HALF) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t p = __shfl_sync(0xffffffffu, b[m], partner);
            if (turns) {
              o[2 * m] = fmaf(o[2 * m], cs[2 * m], -__uint_as_float(p << 16) * sn[2 * m]);
              o[2 * m + 1] = fmaf(o[2 * m + 1], cs[2 * m + 1], -__uint_as_float(p & 0xFFFF0000u) * sn[2 * m + 1]);
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
      if (kind == 0) {
        if (in) __stcs(static_cast<uint4*>(r.q_out) + static_cast<int64_t>(t) * r.q_out_stride / 8 + static_cast<int64_t>(h) * per_head + e, pack_bf16x8(o));
      } else {
        uint8_t scale;
        const uint2 c = mx_codes8(o, E2M1, scale);  // from the rotated fp32 values: one rounding
        if (in) {
          const int64_t at = (row0 + static_cast<int64_t>(h) * a.page_size) * per_head + e;
          uint8_t* const codes = kind == 1 ? a.k_codes : a.v_codes;
          if (E2M1) reinterpret_cast<uint32_t*>(codes)[at] = c.x;
          else reinterpret_cast<uint2*>(codes)[at] = c;
          if ((lane & 3) == 0) (kind == 1 ? a.k_scales : a.v_scales)[at / 4] = scale;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) x[i] = next[i];
  }
}

// Warps that share a token: as many as its groups of heads allow while the tokens alone
// leave SMs idle.
int token_parts(const RopeArgs& r) {
  const int together = 32 / (r.kv.head_dim / 8);
  const int units = (r.n_q_heads + together - 1) / together + 2 * ((r.kv.n_heads + together - 1) / together);
  int parts = 1;
  while (parts < 16 && 2 * parts * kUnroll <= units + kUnroll && static_cast<int64_t>(r.kv.T) * parts < 152 * 32) parts *= 2;
  return parts;
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeArgs& r, cudaStream_t s) {
  const int parts = token_parts(r);
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
