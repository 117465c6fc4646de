// What the two attention kernels share: the work list and how it is split.
//
// Work is counted in units of kUnit keys of one (sequence, KV head, row tile);
// a row is one (new token, query head of the KV head's group), token-major, so
// a KV head's keys are read once for all its query heads.  The units of the
// whole batch lie on one line (sequence, then KV head, then row tile, then
// keys) and every CTA takes an equal stretch of it, found from the lengths on
// the device: ragged batches stay balanced and the host needs no lengths.  A
// stretch ends inside at most two segments (a segment is one row tile's keys);
// those leave their accumulator and softmax statistics in the workspace, and
// the last CTA to arrive at a segment joins its parts, always in key order, so
// results do not depend on which one that is.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace mxk {

struct AttnSeq {
  int q0, n, kv, tiles;  // first token, new tokens, keys, row tiles (0: nothing to do here)
};

struct AttnTile {
  int lo, hi;  // keys [lo, hi) that some row of the tile sees (lo == hi: none)
  int first;   // lo rounded down to the unit
  int units;   // at least 1: a tile without keys still writes its rows
};

// Sequence b as this launch handles it: only sequences of more than
// a.rows_above and at most a.rows_upto rows; bad metadata sets the status word
// (where `report`) and leaves nothing to do.
template <int kRows>
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b, bool report) {
  AttnSeq s;
  s.q0 = a.q_starts[b];
  const int end = a.q_starts[b + 1];
  s.kv = a.kv_lens[b];
  s.n = end - s.q0;
  s.tiles = 0;
  if (s.q0 < 0 || end < s.q0 || end > a.T || s.n > a.max_q_len || s.kv < 0 ||
      s.kv > static_cast<int64_t>(a.max_pages) * a.page_size) {
    if (report) set_status(a.status, MX_ERR_DEVICE_ARG);
    s.n = 0;
    return s;
  }
  const int rows = s.n * a.group;
  if (rows > a.rows_above && rows <= a.rows_upto) s.tiles = (rows + kRows - 1) / kRows;
  return s;
}

template <int kRows, int kUnit>
__device__ __forceinline__ AttnTile attn_tile(const AttnArgs& a, const AttnSeq& s, int tile) {
  AttnTile t;
  t.lo = 0;
  t.hi = s.kv;
  const int base = s.kv - s.n;  // the position of the first new token
  if (a.causal) {
    const int last = min(((tile + 1) * kRows - 1) / a.group, s.n - 1);
    t.hi = min(s.kv, max(base + last + 1, 0));
  }
  if (a.window > 0) {
    // in 64 bits: base may be negative and the window as large as an int
    const int64_t lo = static_cast<int64_t>(base) + tile * kRows / a.group + 1 - a.window;
    t.lo = static_cast<int>(lo < 0 ? 0 : lo);
  }
  t.lo = min(t.lo, t.hi);
  t.first = t.lo / kUnit * kUnit;
  t.units = max((t.hi - t.first + kUnit - 1) / kUnit, 1);
  return t;
}

// Units of one KV head of a sequence.
template <int kRows, int kUnit>
__device__ __forceinline__ int attn_seq_units(const AttnArgs& a, const AttnSeq& s) {
  int u = 0;
  for (int t = 0; t < s.tiles; ++t) u += attn_tile<kRows, kUnit>(a, s, t).units;
  return u;
}

// A CTA's stretch [u, end) of the line and the sequence that holds u, with u's
// place inside that sequence.
struct AttnShare {
  int64_t total;
  int ctas;        // CTAs that have a stretch
  int64_t u, end;
  int seq;
  int64_t in_seq;
};

// The CTA whose stretch holds unit u: the largest c with total * c / ctas <= u.
__device__ __forceinline__ int attn_cta_of(int64_t u, int64_t total, int ctas) {
  return static_cast<int>(((u + 1) * ctas - 1) / total);
}
__device__ __forceinline__ int64_t attn_start_of(int c, int64_t total, int ctas) { return total * c / ctas; }

// Block-wide; kThreads threads call it, scratch holds kThreads / 32 + 4 words.
template <int kRows, int kUnit, int kThreads>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a, int64_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = kThreads / 32;
  AttnShare r;
  // the line's length
  int64_t mine = 0, first_units = 0;
  for (int b = tid; b < a.n_seqs; b += kThreads) {
    const AttnSeq s = attn_seq<kRows>(a, b, blockIdx.x == 0);
    const int64_t u = static_cast<int64_t>(attn_seq_units<kRows, kUnit>(a, s)) * a.n_kv_heads;
    if (b == tid) first_units = u;
    mine += u;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  if (lane == 0) scratch[warp] = mine;
  __syncthreads();
  r.total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) r.total += scratch[w];
  __syncthreads();
  int64_t n = (r.total + a.min_units - 1) / a.min_units;
  r.ctas = static_cast<int>(n < gridDim.x ? n : gridDim.x);
  r.seq = 0;
  r.in_seq = 0;
  r.u = r.end = 0;
  if (static_cast<int>(blockIdx.x) >= r.ctas) return r;
  r.u = attn_start_of(blockIdx.x, r.total, r.ctas);
  r.end = attn_start_of(blockIdx.x + 1, r.total, r.ctas);
  // the sequence that holds u: inclusive scans of kThreads sequences at a time
  int64_t before = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
    const int b = b0 + tid;
    int64_t v = first_units;
    if (b0 > 0) {
      v = 0;
      if (b < a.n_seqs) {
        const AttnSeq s = attn_seq<kRows>(a, b, false);
        v = static_cast<int64_t>(attn_seq_units<kRows, kUnit>(a, s)) * a.n_kv_heads;
      }
    }
    int64_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t all = 0, below = before;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) below += scratch[w];
      all += scratch[w];
    }
    const int64_t from = below + incl - v;
    if (v > 0 && from <= r.u && r.u < from + v) {
      scratch[kW] = b;
      scratch[kW + 1] = r.u - from;
    }
    before += all;
    const bool found = r.u < before;
    __syncthreads();
    if (found) break;
  }
  r.seq = static_cast<int>(scratch[kW]);
  r.in_seq = scratch[kW + 1];
  __syncthreads();
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace mxk
