// What the two attention kernels share: the work list and how it is split.
//
// Work is counted in units of kUnit keys of one (sequence, KV head, row tile);
// a row is one (new token, query head of the KV head's group), token-major, so
// a KV head's keys are read once for all its query heads.  The units of the
// whole batch lie on one line (sequence, then KV head, then row tile, then
// keys) and every CTA takes an equal stretch of it, found from the lengths on
// the device: ragged batches stay balanced and the host needs no lengths.  In
// front of each segment's units the line has kCost places that hold no work:
// what a segment costs beside its keys (its queries, its output), in units, so
// that a CTA with many short segments gets fewer keys.  A stretch ends inside at
// most two segments (a segment is one row tile's keys); those leave their
// accumulator and softmax statistics in the workspace, and the last CTA to arrive
// at a segment joins its parts, always in key order, so results do not depend on
// which one that is.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

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
//
// This and what else runs once a segment or less is not inlined: its copies
// would push the unit loops out of the instruction caches, and make a kernel's
// first pass wait for its code.
template <int kRows>
__device__ __noinline__ AttnSeq attn_seq(const AttnArgs& a, int b, bool report) {
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
__device__ __noinline__ AttnTile attn_tile(const AttnArgs& a, const AttnSeq& s, int tile) {
  AttnTile t;
  t.lo = 0;
  t.hi = s.kv;
  const int base = s.kv - s.n;  // the position of the first new token
  if (a.causal) {
    const int last = min(a.group_div.of((tile + 1) * kRows - 1), s.n - 1);
    t.hi = min(s.kv, max(base + last + 1, 0));
  }
  if (a.window > 0) {
    // in 64 bits: base may be negative and the window as large as an int
    const int64_t lo = static_cast<int64_t>(base) + a.group_div.of(tile * kRows) + 1 - a.window;
    t.lo = static_cast<int>(lo < 0 ? 0 : lo);
  }
  t.lo = min(t.lo, t.hi);
  t.first = t.lo / kUnit * kUnit;
  t.units = max((t.hi - t.first + kUnit - 1) / kUnit, 1);
  return t;
}

// The first key that a row at position `at` sees with a window.  The position may be
// negative (more new tokens than keys) and the window as large as an int, so they are
// compared before the difference is taken.
__device__ __forceinline__ int attn_row_lo(const AttnArgs& a, int at) { return at >= a.window ? at - a.window + 1 : 0; }

// Places on the line of one KV head of a sequence; kWarp: the lanes of a warp
// (all with the same sequence) take the tiles in turn.
template <int kRows, int kUnit, int kCost, bool kWarp>
__device__ __forceinline__ int attn_seq_places(const AttnArgs& a, const AttnSeq& s) {
  int u = 0;
  for (int t = kWarp ? threadIdx.x & 31 : 0; t < s.tiles; t += kWarp ? 32 : 1)
    u += attn_tile<kRows, kUnit>(a, s, t).units + kCost;
  return kWarp ? __reduce_add_sync(0xffffffffu, u) : u;
}

// A CTA's stretch [u, end) of the line; the line's first `longer` stretches have
// `each` + 1 places, the others `each`.  Places are 32-bit, and those of one KV head
// a signed int: the host refuses what could have more.
struct AttnShare {
  uint32_t total;
  int ctas;             // CTAs that have a stretch
  uint32_t each, longer;
  uint32_t u, end;
  int seq;              // the sequence that holds u,
  uint32_t in_seq;      // and u's place in it

  __device__ __forceinline__ uint32_t start_of(uint32_t c) const { return c * each + min(c, longer); }
  // the CTA whose stretch holds place v
  __device__ __forceinline__ int cta_of(uint32_t v) const {
    const uint32_t head = longer * (each + 1);
    return static_cast<int>(v < head ? v / (each + 1) : longer + (v - head) / each);
  }
};

constexpr int kAttnScan = 128;  // sequences looked at together

// Block-wide (kThreads threads); `units` holds kAttnScan words.  kWarp: a warp
// counts a sequence of several tiles (long ones have hundreds), else a thread.
template <int kRows, int kUnit, int kCost, int kThreads, bool kWarp>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a, uint32_t* units) {
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr int kPer = kAttnScan / 32;
  AttnShare r;
  uint64_t all_of_them = 0;
  r.seq = 0;
  r.in_seq = r.u = r.end = 0;
  uint32_t v[kPer], mine = 0, before = 0;
  // Once over all sequences for the line's length, then again for the one that
  // holds u; with one scan's worth of sequences the second pass has them.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < a.n_seqs; b0 += kAttnScan) {
      if (pass == 0 || a.n_seqs > kAttnScan) {
        // a thread a sequence, and then a warp each of those with several tiles
        // (kWarp), which are marked
        constexpr uint32_t kLong = ~0u;
        for (int i = tid; i < kAttnScan; i += kThreads) {
          uint32_t u = 0;
          if (b0 + i < a.n_seqs) {
            const AttnSeq s = attn_seq<kRows>(a, b0 + i, pass == 0 && blockIdx.x == 0);
            if (kWarp && s.tiles > 1) u = kLong;
            else u = static_cast<uint32_t>(attn_seq_places<kRows, kUnit, kCost, false>(a, s)) * a.n_kv_heads;
          }
          units[i] = u;
        }
        __syncthreads();
        if (kWarp) {
          for (int i = tid / 32; i < kAttnScan && b0 + i < a.n_seqs; i += kThreads / 32) {
            if (units[i] != kLong) continue;
            const AttnSeq s = attn_seq<kRows>(a, b0 + i, false);
            const uint32_t u = static_cast<uint32_t>(attn_seq_places<kRows, kUnit, kCost, true>(a, s)) * a.n_kv_heads;
            if (lane == 0) units[i] = u;
          }
          __syncthreads();
        }
        mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += v[i] = units[lane * kPer + i];
        __syncthreads();
        if (pass == 0) {
          // in two halves, which a warp's sums hold
          uint32_t lo = 0, hi = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) lo += v[i] & 0xFFFFu, hi += v[i] >> 16;
          all_of_them += __reduce_add_sync(0xffffffffu, lo) + (static_cast<uint64_t>(__reduce_add_sync(0xffffffffu, hi)) << 16);
          continue;
        }
      }
      uint32_t incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      uint32_t from = before + incl - mine;
      int at = -1;
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (r.u >= from && r.u - from < v[i]) {
          at = b0 + lane * kPer + i;
          in = r.u - from;
        }
        from += v[i];
      }
      before += all;
      const unsigned hit = __ballot_sync(0xffffffffu, at >= 0);
      if (hit && r.end > r.u) {
        const int src = __ffs(hit) - 1;
        r.seq = __shfl_sync(0xffffffffu, at, src);
        r.in_seq = __shfl_sync(0xffffffffu, in, src);
      }
    }
    if (pass == 0) {
      // The host has refused what the sizes allow to be more than the line holds;
      // starts that fall and rise again may give the same tokens to many sequences.
      r.total = static_cast<uint32_t>(all_of_them);
      if (all_of_them > 4000000000ull) {
        r.total = 0;
        if (blockIdx.x == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
      }
      const uint32_t n = (r.total + a.min_units - 1) / a.min_units;
      r.ctas = static_cast<int>(min(n, gridDim.x));
      r.each = r.ctas > 0 ? r.total / r.ctas : 1;
      r.longer = r.total - r.each * r.ctas;
      if (blockIdx.x < static_cast<unsigned>(r.ctas)) {
        r.u = r.start_of(blockIdx.x);
        r.end = r.start_of(blockIdx.x + 1);
      }
    }
  }
  return r;
}

// Between CTAs' stretches a segment of `units` units is split before unit k only
// for before <= k <= units - behind: a part of fewer than kSnap units costs more
// than it saves, and goes to the neighbour.
template <int kSnap>
struct AttnSplit {
  int before, behind;
  __device__ __forceinline__ explicit AttnSplit(int units) {
    before = kSnap == 1 ? 1 : min(kSnap, (units + 1) / 2);
    behind = kSnap == 1 ? 1 : min(kSnap, units + 1 - before);
  }
};

// Where a CTA is on the line: a segment (one row tile of one KV head of one
// sequence) and the unit `place` of it (below zero: the places without work).
template <int kRows, int kUnit, int kCost, int kSnap>
struct AttnCursor {
  uint32_t u, end;  // on the line
  int b, head, tile, place;
  AttnSeq s;
  AttnTile t;

  // At the share's first unit; whole warps call it.
  template <bool kWarp>
  __device__ __forceinline__ void start(const AttnArgs& a, const AttnShare& share) {
    u = share.u;
    end = share.end;
    b = share.seq;
    head = tile = place = 0;
    if (u >= end) return;
    s = attn_seq<kRows>(a, b, false);
    const int per_head = attn_seq_places<kRows, kUnit, kCost, kWarp>(a, s);
    head = static_cast<int>(share.in_seq / max(per_head, 1));
    place = static_cast<int>(share.in_seq - static_cast<uint32_t>(head) * per_head);
    if (kWarp) {
      const int lane = threadIdx.x & 31;
      for (; tile < s.tiles; tile += 32) {
        const int n = tile + lane < s.tiles ? attn_tile<kRows, kUnit>(a, s, tile + lane).units + kCost : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, place < incl);
        if (hit) {
          const int src = __ffs(hit) - 1;
          place -= __shfl_sync(0xffffffffu, incl - n, src);
          tile += src;
          break;
        }
        place -= __shfl_sync(0xffffffffu, incl, 31);
      }
      t = attn_tile<kRows, kUnit>(a, s, tile);
    } else {
      t = attn_tile<kRows, kUnit>(a, s, 0);
      while (place >= t.units + kCost && tile + 1 < s.tiles) {
        place -= t.units + kCost;
        t = attn_tile<kRows, kUnit>(a, s, ++tile);
      }
    }
    place -= kCost;
    if (kSnap > 1 && place > 0 && place < t.units) {
      const AttnSplit<kSnap> split(t.units);
      const int to = place < split.before ? 0 : place > t.units - split.behind ? t.units : place;
      u += to - place;
      place = to;
    }
  }

  // Past what has no work: to a unit of the stretch, or false where it has no
  // more.
  __device__ __forceinline__ bool settle(const AttnArgs& a) {
    while (u < end) {
      if (place < 0) {
        const int d = static_cast<int>(min(static_cast<uint32_t>(-place), end - u));
        u += d;
        place += d;
        continue;
      }
      if (place < t.units) {
        const int k = place + static_cast<int>(end - u);  // the next stretch's first unit, where that lies in the segment
        if (kSnap == 1 || k >= t.units || k >= AttnSplit<kSnap>(t.units).before) return true;
        u = end;
        return false;
      }
      place = -kCost;
      if (++tile == s.tiles) {
        tile = 0;
        if (++head == a.n_kv_heads) {
          head = 0;
          do {
            if (++b >= a.n_seqs) return false;
            s = attn_seq<kRows>(a, b, false);
          } while (s.tiles == 0);
        }
      }
      t = attn_tile<kRows, kUnit>(a, s, tile);
    }
    return false;
  }
  // Units of the segment from `place` on that lie in the stretch, and past them.
  __device__ __forceinline__ int take() const {
    if (kSnap == 1) return static_cast<int>(min(static_cast<uint32_t>(t.units - place), end - u));
    const int k = place + static_cast<int>(min(end - u, static_cast<uint32_t>(t.units)));
    return (k > t.units - AttnSplit<kSnap>(t.units).behind ? t.units : k) - place;
  }
  __device__ __forceinline__ void pass(int n) {
    u += n;
    place += n;
  }
};

// Where a unit's keys lie in the cache, for the warp that fetches them: 16-key
// groups, group = lane % (kUnit / 16), in boxes of a.box_keys keys.
template <int kUnit>
struct AttnWalk {
  static constexpr int kGroups = kUnit / 16;
  const int32_t* table;
  int entry, off;     // the group's first key: entry of the table, place in the page
  int lo, hi;         // the keys to read, counted from the unit's first
  int window, pages;  // 32 entries of the table from `window` on, one a lane

  template <class Cursor>
  __device__ __forceinline__ void start(const AttnArgs& a, const Cursor& c, int group) {
    table = a.block_table + static_cast<int64_t>(c.b) * a.max_pages;
    const int first = c.t.first + c.place * kUnit;
    entry = a.page_div.of(first + 16 * group);
    off = first + 16 * group - entry * a.page_size;
    lo = c.t.lo - first;
    hi = c.t.hi - first;
    window = -64;
    pages = 0;
  }
  // The group's box: its first cache row, or -1 where it has no page or no key
  // to read; `here`: the groups (a bit each) that are there, `bad`: those whose
  // page is not one, which is reported.
  __device__ __forceinline__ int box(const AttnArgs& a, int head, int group, uint32_t& here, uint32_t& bad) {
    if (__any_sync(0xffffffffu, entry - window >= 32)) {
      window = __shfl_sync(0xffffffffu, entry, 0);
      pages = __ldg(table + min(window + static_cast<int>(threadIdx.x & 31), a.max_pages - 1));
    }
    const int page = __shfl_sync(0xffffffffu, pages, entry - window);
    const bool seen = 16 * group < hi && 16 * group + 16 > lo;
    const bool there = seen && page >= 0 && page < a.num_pages;
    if (seen && !there) set_status(a.status, MX_ERR_DEVICE_ARG);
    here = __ballot_sync(0xffffffffu, there) & ((1u << kGroups) - 1);
    bad = __ballot_sync(0xffffffffu, seen && !there) & ((1u << kGroups) - 1);
    const bool some = (here >> group & ((1u << (a.box_keys / 16)) - 1)) != 0;
    return some ? (page * a.n_kv_heads + head) * a.page_size + off : -1;
  }
  __device__ __forceinline__ void step(const AttnArgs& a) {
    lo -= kUnit, hi -= kUnit;
    for (off += kUnit; off >= a.page_size; off -= a.page_size) ++entry;
  }
};

// How a segment of `units` units, its first at place `seg` of the line, is
// shared out: its parts lie with CTAs first .. first + parts - 1.
struct AttnParts {
  int first, parts;
};
template <int kSnap>
__device__ __forceinline__ AttnParts attn_parts(const AttnShare& sh, uint32_t seg, int units) {
  const AttnSplit<kSnap> split(units);
  AttnParts p;
  p.first = sh.cta_of(seg + split.before - 1);
  p.parts = sh.cta_of(seg + units - split.behind) - p.first + 1;
  return p;
}
// The workspace slot of a CTA's part: the part that begins a segment and those
// that continue one lie apart (a CTA has at most one of each that is not whole).
__device__ __forceinline__ int attn_slot(int cta, bool begins) { return 2 * cta + (begins ? 1 : 0); }

// One more part of a segment is there; returns how many were before it.  What the
// block wrote ahead of a barrier is seen by whoever finds it the last, and what
// the others wrote by the block behind the next barrier.
__device__ __forceinline__ unsigned attn_arrive(unsigned* counter) {
  unsigned before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  return before;
}

// A wait for an mbarrier's phase.  One that runs out sets the status word and
// makes every later wait of the CTA (`failed` in its shared memory) give up at
// once.  With kNow a limit of zero waits for nothing: a try suspends the thread for
// longer than the few-rows kernel's ordinary waits, which would never run out.
template <bool kNow>
__device__ __noinline__ bool attn_wait_long(volatile int* failed, uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                                   int* status) {
  const uint64_t t0 = globaltimer_ns();
  const bool now = kNow && limit_ns == 0;
  for (uint32_t n = 1; now || !mbar_try_wait(bar, parity); ++n) {
    if (!now && (n & 15u)) continue;
    if (*failed) return false;
    if (now || globaltimer_ns() - t0 > limit_ns) {
      *failed = 1;
      set_status(status, MX_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
template <bool kNow>
__device__ __forceinline__ bool attn_wait(volatile int* failed, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  const uint32_t b = smem_u32(bar);
  const bool there = kNow && a.wait_limit_ns == 0 ? mbar_test_wait(b, parity) : mbar_try_wait(b, parity);
  if (__builtin_expect(there, 1)) return true;
  return attn_wait_long<kNow>(failed, b, parity, a.wait_limit_ns, a.status);
}

// A stage of a ring and the parity of its current round.
template <int kN>
struct Ring {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kN) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// One arrival for a warp's lanes, behind whatever each of them did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(bar));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Tensor map of a code table, a.box_keys rows a box, swizzled so that 16-byte
// pieces of neighbouring rows lie in different banks (or not at all).
inline cudaError_t attn_code_map(CUtensorMap* map, const AttnArgs& a, const uint8_t* codes, int row_bytes, bool swizzle) {
  // atomic: the first calls may come from several threads, which find the same
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 encode = known.load(std::memory_order_relaxed);
  if (!encode) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    known.store(encode, std::memory_order_relaxed);
  }
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(a.num_pages) * a.n_kv_heads * a.page_size};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(row_bytes), static_cast<cuuint32_t>(a.box_keys)}, es[2] = {1, 1};
  const CUtensorMapSwizzle sw = !swizzle           ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : row_bytes == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_32B;
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace mxk
