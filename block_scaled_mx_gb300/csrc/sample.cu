// A token from a row of logits by temperature, top-k, top-p and min-p and one given
// random number, by the inverse of the distribution function in the order of the
// tokens' numbers.
//
// A cluster of CTAs holds the row in its shared memory (read once) and goes over it a
// few times from there:
//   1. the row's maximum m;
//   2. with top-k or top-p, a histogram of counts and weights over bins of m - logit,
//      merged across the cluster slice by slice.  The bin in which the kept prefix ends
//      holds few tokens as a rule; they are ranked one against the other.  Where it
//      holds many, it is divided by the bits of the logit until few are left or all of
//      them are equal (then the first ones by number are kept);
//   3. the kept weights, by warp; the warp in which the random number falls goes over
//      its stretch once more.
//
// Weights are whole numbers, 2^43 e^((logit - m) / temperature) rounded down, so sums
// are exact in any order (no atomic changes a result) and two calls agree.  A draw next
// to a token's border is decided by the weights' own rounding: e^x is taken in two floats
// with a table of 2^(j/64), 2^-31 off where one float's exponential would be 2^-22, as a
// vocabulary has 10^5 borders.  Weights below 2^-44 of the largest are zero.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <climits>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace mxk {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kDigit = 10;  // bins of a histogram, bits of the logit that one divides by
constexpr int kCandidates = 256;          // ranked one against the other
constexpr int kMaxCluster = 8;
constexpr int kOneBits = 43;
constexpr unsigned long long kOne = 1ull << kOneBits;  // the largest weight; 2^20 of them fit 64 bits

// 2^(j/64) as the sum of two floats.
__constant__ float2 kExp2[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},
};

// Where the kept prefix ends: the bin, what lies before it, what it holds.
struct Found {
  int bin;
  uint32_t before, count;
  unsigned long long before_mass;
};
// The end itself: tokens above `key`, and the first `quota` of those with it.
struct End {
  uint32_t key, quota;
  unsigned long long mass;  // of all of them
};

struct Control {
  float c_hi, c_lo;
  float max[kMaxCluster];
  int nan[kMaxCluster];
  uint32_t first[kMaxCluster];  // lowest place of the maximum
  uint32_t slice_count[2][kMaxCluster];
  unsigned long long slice_mass[2][kMaxCluster];
  Found found;
  End end;
  uint32_t key_min[kMaxCluster], key_max[kMaxCluster];
  uint32_t n;  // candidates (rank 0)
  uint32_t cand_key[kCandidates], cand_at[kCandidates];
  unsigned long long cand_mass[kCandidates];
  uint32_t warp_eq[kMaxCluster * kWarps];
  unsigned long long warp_mass[kMaxCluster * kWarps];
  int hit_warp;
  uint32_t hit_eq;
  unsigned long long hit_before, total, target;
  uint32_t red[kWarps], red2[kWarps];
  unsigned long long red64[kWarps];
  float2 exp2_table[64];
  uint32_t hist_count[kBins], hist_lo[kBins], hist_hi[kBins];
};

// Logits in their order as unsigned numbers (both zeros the same), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// 2^43 e^((x - max) / temperature), rounded down; c_hi + c_lo = log2(e) / temperature.
__device__ __forceinline__ unsigned long long weight_of(float x, float max, float c_hi, float c_lo, const float2* table) {
  if (x == max) return kOne;
  const float s = x - max;
  const float t = s * c_hi;
  if (!(t > -44.0f)) return 0ull;  // also -inf, and NaN of an infinite maximum
  // x - max = s + e exactly (the error of a sum of two floats), its product likewise
  const float v = s - x;
  const float e = (x - (s - v)) - (max + v);
  const float t_lo = fmaf(s, c_hi, -t) + fmaf(s, c_lo, e * c_hi);
  const float shifted = t + 196608.0f;  // 1.5 * 2^17: the sum's last place is 2^-6
  const int j = __float_as_int(shifted) - 0x48400000;
  const float f = (t - (shifted - 196608.0f)) + t_lo;
  // 2^f - 1 for |f| <= 2^-7: the next term is below 2^-44
  const float q = f * fmaf(f, fmaf(f, fmaf(f, 9.6181291e-3f, 5.5504109e-2f), 0.24022651f), 0.69314718f);
  const float2 p = table[j & 63];
  const float lo = fmaf(p.x, q, p.y);  // below 2^-6 in size
  const unsigned long long whole = static_cast<unsigned long long>((__float_as_uint(p.x) & 0x7FFFFFu) | 0x800000u) << (kOneBits - 23);
  const long long part = static_cast<long long>(__float2int_rn(lo * 0x1p36f)) << (kOneBits - 36);
  return (whole + part) >> -(j >> 6);
}

template <bool BF16>
__device__ __forceinline__ float element(const uint4& v, int m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (!BF16) return __uint_as_float(w[m]);
  return __uint_as_float(m & 1 ? w[m / 2] & 0xFFFF0000u : w[m / 2] << 16);
}

__device__ __forceinline__ unsigned long long shfl_up64(unsigned long long v, int d) {
  return __shfl_up_sync(0xffffffffu, v, d);
}

// The row's segment of this CTA and what is known of the row.
template <bool BF16>
struct Row {
  static constexpr int VE = BF16 ? 8 : 4;  // elements of 16 bytes
  const uint4* seg;
  int vecs;           // of the segment
  uint32_t at0;       // place of its first element
  float max, c_hi, c_lo, bin_scale;
  const float2* table;
  __device__ __forceinline__ unsigned long long weight(float x) const { return weight_of(x, max, c_hi, c_lo, table); }
  // Bins of the first histogram: more for lower logits, by a function that keeps order.
  __device__ __forceinline__ int bin(float x) const {
    return x == max ? 0 : min(kBins - 1, __float2int_rz((max - x) * bin_scale));
  }
};

// Tokens of bin `bin0` whose keys agree with `prefix` above `shift` (32: all of the bin).
struct Subset {
  int bin0;
  int shift;
  uint32_t prefix;
  template <bool BF16>
  __device__ __forceinline__ bool holds(const Row<BF16>& r, float x, uint32_t key) const {
    return r.bin(x) == bin0 && (shift >= 32 || (key >> shift) == prefix);
  }
};

// Histogram of the whole row (level 0) or of a subset by the `kDigit` bits below its
// shift, highest first; merged in slices of kBins / C bins, one a CTA, and the slices'
// sums known to all.
template <bool BF16>
__device__ void histogram(const Row<BF16>& r, Control& ctl, uint32_t* slice_count, unsigned long long* slice_mass, bool masses,
                          int level, const Subset& sub) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  for (int b = tid; b < kBins; b += kThreads) ctl.hist_count[b] = ctl.hist_lo[b] = ctl.hist_hi[b] = 0u;
  __syncthreads();
  const int low = sub.shift - kDigit;  // the digit's lowest bit (may be negative: fewer bits left)
  // the last bin, which may hold nearly all of a row, is added up in registers
  uint32_t last_count = 0;
  unsigned long long last_mass = 0;
  auto add = [&](int b, unsigned long long w) {
    const uint32_t lo = static_cast<uint32_t>(w);
    const uint32_t hi = static_cast<uint32_t>(w >> 32) + (atomicAdd(&ctl.hist_lo[b], lo) > ~lo ? 1u : 0u);
    if (hi) atomicAdd(&ctl.hist_hi[b], hi);
  };
  for (int i = tid; i < r.vecs; i += kThreads) {
    const uint4 v = r.seg[i];
#pragma unroll
    for (int m = 0; m < Row<BF16>::VE; ++m) {
      const float x = element<BF16>(v, m);
      int b;
      if (level == 0) {
        b = r.bin(x);
      } else {
        const uint32_t key = key_of(x);
        if (!sub.holds(r, x, key)) continue;
        const uint32_t digit = low >= 0 ? (key >> low) & (kBins - 1) : (key << -low) & (kBins - 1);
        b = kBins - 1 - static_cast<int>(digit);
      }
      const unsigned long long w = masses ? r.weight(x) : 0ull;
      if (b == kBins - 1) {
        ++last_count;
        last_mass += w;
      } else {
        atomicAdd(&ctl.hist_count[b], 1u);
        if (w) add(b, w);
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    last_count += __shfl_xor_sync(0xffffffffu, last_count, d);
    last_mass += __shfl_xor_sync(0xffffffffu, last_mass, d);
  }
  if (lane == 0 && last_count) {
    atomicAdd(&ctl.hist_count[kBins - 1], last_count);
    add(kBins - 1, last_mass);
  }
  cluster.sync();
  const int S = kBins / C;
  uint32_t count = 0;
  unsigned long long mass = 0;
  for (int b = tid; b < S; b += kThreads) {
    uint32_t n = 0;
    unsigned long long w = 0;
    for (int c = 0; c < C; ++c) {
      const Control* peer = cluster.map_shared_rank(&ctl, c);
      const int at = R * S + b;
      n += peer->hist_count[at];
      if (masses) w += (static_cast<unsigned long long>(peer->hist_hi[at]) << 32) + peer->hist_lo[at];
    }
    slice_count[b] = n;
    slice_mass[b] = w;
    count += n;
    mass += w;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    count += __shfl_xor_sync(0xffffffffu, count, d);
    mass += __shfl_xor_sync(0xffffffffu, mass, d);
  }
  if (lane == 0) {
    ctl.red[warp] = count;
    ctl.red64[warp] = mass;
  }
  __syncthreads();
  if (tid < C) {
    uint32_t n = 0;
    unsigned long long w = 0;
    for (int i = 0; i < kWarps; ++i) {
      n += ctl.red[i];
      w += ctl.red64[i];
    }
    Control* peer = cluster.map_shared_rank(&ctl, tid);
    peer->slice_count[level ? 1 : 0][R] = n;
    peer->slice_mass[level ? 1 : 0][R] = w;
  }
  cluster.sync();
}

// The bin in which the `target`th token, or unit of weight, lies; the sums of what is
// before the histogram's tokens are in `base`.
__device__ Found find_bin(Control& ctl, const uint32_t* slice_count, const unsigned long long* slice_mass, bool by_mass,
                          unsigned long long target, int which, const Found& base) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), R = cluster.block_rank(), lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    uint32_t n = base.before;
    unsigned long long w = base.before_mass;
    int owner = 0;
    for (; owner < C - 1; ++owner) {
      const uint32_t n2 = n + ctl.slice_count[which][owner];
      const unsigned long long w2 = w + ctl.slice_mass[which][owner];
      if ((by_mass ? w2 : n2) >= target) break;
      n = n2;
      w = w2;
    }
    if (owner == R) {
      // each lane a run of the slice's bins, then the lane whose run holds the target
      const int S = kBins / C, per = S / 32;
      uint32_t run = 0;
      unsigned long long run_mass = 0;
      for (int i = 0; i < per; ++i) {
        run += slice_count[lane * per + i];
        run_mass += slice_mass[lane * per + i];
      }
      uint32_t in = run;
      unsigned long long in_mass = run_mass;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, in, d);
        const unsigned long long z = shfl_up64(in_mass, d);
        if (lane >= d) {
          in += y;
          in_mass += z;
        }
      }
      const bool reached = (by_mass ? w + in_mass : static_cast<unsigned long long>(n + in)) >= target;
      const unsigned hits = __ballot_sync(0xffffffffu, reached);
      if (lane == (hits ? __ffs(hits) - 1 : 31)) {
        n += in - run;
        w += in_mass - run_mass;
        int i = 0;
        for (; i < per - 1; ++i) {
          const uint32_t n2 = n + slice_count[lane * per + i];
          const unsigned long long w2 = w + slice_mass[lane * per + i];
          if ((by_mass ? w2 : n2) >= target) break;
          n = n2;
          w = w2;
        }
        const Found f{R * S + lane * per + i, n, slice_count[lane * per + i], w};
        for (int c = 0; c < C; ++c) {
          Control* peer = cluster.map_shared_rank(&ctl, c);
          peer->found = f;
          if (c == 0) peer->n = 0u;
        }
      }
    }
  }
  cluster.sync();
  return ctl.found;
}

// Where the prefix of `target` tokens (or of tokens until their weights reach target)
// ends, from the level-0 histogram on.
template <bool BF16>
__device__ End find_end(const Row<BF16>& r, Control& ctl, uint32_t* const (&slice_count)[2], unsigned long long* const (&slice_mass)[2],
                        bool by_mass, bool masses, unsigned long long target) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  Found f = find_bin(ctl, slice_count[0], slice_mass[0], by_mass, target, 0, Found{});
  Subset sub{f.bin, 32, 0u};
  while (true) {
    // the subset's least and largest key, and its tokens where they are few
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    Control* leader = cluster.map_shared_rank(&ctl, 0);
    for (int i = tid; i < r.vecs; i += kThreads) {
      const uint4 v = r.seg[i];
#pragma unroll
      for (int m = 0; m < Row<BF16>::VE; ++m) {
        const float x = element<BF16>(v, m);
        if (r.bin(x) != sub.bin0) continue;
        const uint32_t key = key_of(x);
        if (sub.shift < 32 && (key >> sub.shift) != sub.prefix) continue;
        lo = min(lo, key);
        hi = max(hi, key);
        if (f.count <= kCandidates) {
          const uint32_t at = atomicAdd(&leader->n, 1u);
          if (at < kCandidates) {
            leader->cand_key[at] = key;
            leader->cand_at[at] = r.at0 + static_cast<uint32_t>(i * Row<BF16>::VE + m);
            leader->cand_mass[at] = masses ? r.weight(x) : 0ull;
          }
        }
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      ctl.red[warp] = lo;
      ctl.red2[warp] = hi;
    }
    __syncthreads();
    if (tid < C) {
      for (int i = 0; i < kWarps; ++i) {
        lo = min(lo, ctl.red[i]);
        hi = max(hi, ctl.red2[i]);
      }
      Control* peer = cluster.map_shared_rank(&ctl, tid);
      peer->key_min[R] = lo;
      peer->key_max[R] = hi;
    }
    cluster.sync();
    lo = 0xFFFFFFFFu;
    hi = 0u;
    for (int c = 0; c < C; ++c) {
      lo = min(lo, ctl.key_min[c]);
      hi = max(hi, ctl.key_max[c]);
    }
    if (lo == hi) {  // equal logits: the first ones by number
      const unsigned long long w = masses ? r.weight(value_of(lo)) : 0ull;
      unsigned long long quota = by_mass ? (w ? (target - f.before_mass + w - 1) / w : f.count) : target - f.before;
      if (quota > f.count) quota = f.count;
      return End{lo, static_cast<uint32_t>(quota), f.before_mass + quota * w};
    }
    if (f.count <= kCandidates) {
      if (R == 0) {
        // a token's rank among them: those of a larger logit, or of the same and a lower number
        const int n = static_cast<int>(f.count);
        if (tid < n) {
          const uint32_t key = ctl.cand_key[tid], at = ctl.cand_at[tid];
          uint32_t rank = 0, equal = 0;
          unsigned long long mass = f.before_mass;
          for (int j = 0; j < n; ++j) {
            const uint32_t k2 = ctl.cand_key[j];
            const bool same = k2 == key && ctl.cand_at[j] < at;
            if (k2 > key || same) {
              ++rank;
              mass += ctl.cand_mass[j];
            }
            if (same) ++equal;
          }
          const unsigned long long w = ctl.cand_mass[tid];
          const bool last = by_mass ? mass < target && mass + w >= target : f.before + rank + 1 == target;
          if (last) {
            for (int c = 0; c < C; ++c) cluster.map_shared_rank(&ctl, c)->end = End{key, equal + 1, mass + w};
          }
        }
      }
      cluster.sync();
      return ctl.end;
    }
    // many, and not all equal: by the next bits of the key
    histogram(r, ctl, slice_count[1], slice_mass[1], masses, 1, sub);
    const Found next = find_bin(ctl, slice_count[1], slice_mass[1], by_mass, target, 1, f);
    const int low = sub.shift - kDigit, digit = kBins - 1 - next.bin;
    sub.prefix = sub.shift >= 32 ? digit : low >= 0 ? (sub.prefix << kDigit) | digit : (sub.prefix << sub.shift) | (digit >> -low);
    sub.shift = max(low, 0);
    f = next;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleArgs a, int chunk) {
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int VE = Row<BF16>::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  const int t = blockIdx.x / C;
  uint4* const seg = reinterpret_cast<uint4*>(smem);
  const int per = chunk * kWarps;  // 16-byte pieces of a CTA: a run of `chunk` a warp
  Control& ctl = *reinterpret_cast<Control*>(smem + static_cast<size_t>(per) * 16);
  uint32_t* const slices = reinterpret_cast<uint32_t*>(&ctl + 1);
  const int S = kBins / C;
  unsigned long long* const slice_mass[2] = {reinterpret_cast<unsigned long long*>(slices), reinterpret_cast<unsigned long long*>(slices) + S};
  uint32_t* const slice_count[2] = {slices + 4 * S, slices + 5 * S};

  const float temperature = a.temperature ? a.temperature[t] : 1.0f;
  const int top_k = a.top_k ? a.top_k[t] : 0;
  const float top_p = a.top_p ? a.top_p[t] : 1.0f;
  const float min_p = a.min_p ? a.min_p[t] : 0.0f;

  // ---- the row into shared memory.  A place counts from the 16-byte boundary at or
  // before the row; what lies outside the row is -inf there.
  const uint8_t* const row = static_cast<const uint8_t*>(a.logits) + static_cast<int64_t>(t) * a.stride * (BF16 ? 2 : 4);
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / (BF16 ? 2 : 4));
  const int end = mis + a.V;  // places of the row are [mis, end)
  const uint4* const base = reinterpret_cast<const uint4*>(row - (reinterpret_cast<uintptr_t>(row) & 15));
  const int v0 = R * per;
  float mx = -INFINITY;
  int nan = 0;
  constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;
  constexpr int kUnroll = 8;
  for (int i0 = tid; i0 < per; i0 += kThreads * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads, p0 = (v0 + i) * VE;
      v[u] = make_uint4(kNone, kNone, kNone, kNone);
      if (i < per && p0 < end && p0 + VE > mis) {
        if (p0 >= mis && p0 + VE <= end) {
          v[u] = __ldcs(base + v0 + i);
        } else {  // the row's first or last piece
          uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
          for (int m = 0; m < VE; ++m) {
            if (p0 + m >= mis && p0 + m < end) {
              if (BF16) {
                const uint32_t h = reinterpret_cast<const uint16_t*>(base)[static_cast<int64_t>(v0 + i) * VE + m];
                w[m / 2] = m & 1 ? (w[m / 2] & 0xFFFFu) | (h << 16) : (w[m / 2] & 0xFFFF0000u) | h;
              } else {
                w[m % 4] = reinterpret_cast<const uint32_t*>(base)[static_cast<int64_t>(v0 + i) * VE + m];
              }
            }
          }
          v[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i < per) seg[i] = v[u];
#pragma unroll
      for (int m = 0; m < VE; ++m) {
        const float x = element<BF16>(v[u], m);
        nan |= x != x;
        mx = fmaxf(mx, x);
      }
    }
  }
  if (tid < 64) ctl.exp2_table[tid] = kExp2[tid];
  if (tid == 0) {
    const double c = 1.4426950408889634074 / static_cast<double>(temperature);
    ctl.c_hi = static_cast<float>(c);
    ctl.c_lo = static_cast<float>(c - static_cast<double>(ctl.c_hi));
  }
  const int any_nan = __syncthreads_or(nan);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  if (lane == 0) ctl.red[warp] = __float_as_uint(mx);
  __syncthreads();
  if (tid < C) {
    for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, __uint_as_float(ctl.red[i]));
    Control* peer = cluster.map_shared_rank(&ctl, tid);
    peer->max[R] = mx;
    peer->nan[R] = any_nan;
  }
  cluster.sync();
  bool bad = !(temperature >= 0.0f);
  mx = -INFINITY;
  for (int c = 0; c < C; ++c) {
    mx = fmaxf(mx, ctl.max[c]);
    bad |= ctl.nan[c] != 0;
  }
  bad |= mx == -INFINITY;
  if (bad) {  // the same in every CTA
    if (R == 0 && tid == 0) {
      a.tokens[t] = -1;
      if (a.logp) a.logp[t] = NAN;
      set_status(a.status, MX_ERR_DEVICE_ARG);
    }
    cluster.sync();  // no CTA leaves while another may write here
    return;
  }
  if (temperature == 0.0f || top_k == 1) {
    uint32_t first = UINT_MAX;
    for (int i = tid; i < per; i += kThreads) {
      const uint4 v = seg[i];
#pragma unroll
      for (int m = VE - 1; m >= 0; --m)
        if (element<BF16>(v, m) == mx) first = min(first, static_cast<uint32_t>((v0 + i) * VE + m));
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) ctl.red2[warp] = first;
    __syncthreads();
    if (tid == 0) {
      for (int i = 0; i < kWarps; ++i) first = min(first, ctl.red2[i]);
      cluster.map_shared_rank(&ctl, 0)->first[R] = first;
    }
    cluster.sync();
    if (R == 0 && tid == 0) {
      for (int c = 0; c < C; ++c) first = min(first, ctl.first[c]);
      a.tokens[t] = static_cast<int32_t>(first) - mis;
      if (a.logp) a.logp[t] = 0.0f;
    }
    return;
  }

  Row<BF16> r;
  r.seg = seg;
  r.vecs = per;
  r.at0 = static_cast<uint32_t>(v0) * VE;
  r.max = mx;
  r.c_hi = ctl.c_hi;
  r.c_lo = ctl.c_lo;
  r.table = ctl.exp2_table;
  // the first histogram spans what has weight (e^-30), and eight units of the logits at least
  r.bin_scale = kBins / fmaxf(30.0f * 1.4426950f / r.c_hi, 8.0f);

  // ---- the kept prefix
  const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.0f;
  End kept{0u, UINT_MAX, 0ull};
  if (by_k || by_p) {
    histogram(r, ctl, slice_count[0], slice_mass[0], by_p, 0, Subset{0, 32, 0u});
    unsigned long long mass = 0;
    for (int c = 0; c < C; ++c) mass += ctl.slice_mass[0][c];
    if (by_k) {
      kept = find_end(r, ctl, slice_count, slice_mass, false, by_p, static_cast<unsigned long long>(top_k));
      mass = kept.mass;
    }
    if (by_p) {
      // a token is kept while the weight before it is below p times the whole: the whole
      // numbers below that product are those below its ceiling
      const unsigned long long p = top_p > 0.0f ? static_cast<unsigned long long>(static_cast<double>(top_p) * 0x1p64) : 0ull;
      unsigned long long target = __umul64hi(p, mass) + (p * mass ? 1ull : 0ull);
      if (target == 0) target = 1;
      kept = find_end(r, ctl, slice_count, slice_mass, true, true, target);
    }
  }

  // ---- kept weights by warp (runs of the row in order)
  const unsigned long long least =
      min_p > 0.0f ? static_cast<unsigned long long>(static_cast<double>(fminf(min_p, 1.0f)) * 0x1p43) : 0ull;
  const unsigned long long w_end = r.weight(value_of(kept.key));
  const uint32_t quota = w_end >= least ? kept.quota : 0u;
  unsigned long long mass = 0;
  uint32_t eq = 0;
  for (int i = warp * chunk + lane; i < (warp + 1) * chunk; i += 32) {
    const uint4 v = seg[i];
#pragma unroll
    for (int m = 0; m < VE; ++m) {
      const float x = element<BF16>(v, m);
      const uint32_t key = key_of(x);
      if (key > kept.key) {
        const unsigned long long w = r.weight(x);
        mass += w >= least ? w : 0ull;
      }
      eq += key == kept.key;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, d);
    eq += __shfl_xor_sync(0xffffffffu, eq, d);
  }
  if (lane < C) {
    Control* peer = cluster.map_shared_rank(&ctl, lane);
    peer->warp_mass[R * kWarps + warp] = mass;
    peer->warp_eq[R * kWarps + warp] = eq;
  }
  if (tid == 0) ctl.hit_warp = -1;
  cluster.sync();  // from here on no CTA touches another's memory

  // ---- the warp in whose run the random number falls
  if (warp == 0) {
    constexpr int kPer = kMaxCluster * kWarps / 32;
    const int n = C * kWarps;
    uint32_t eqs[kPer], eq_run = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      eqs[i] = e < n ? ctl.warp_eq[e] : 0u;
      eq_run += eqs[i];
    }
    uint32_t eq_in = eq_run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, eq_in, d);
      if (lane >= d) eq_in += y;
    }
    uint32_t eq_before = eq_in - eq_run;
    unsigned long long ws[kPer], run = 0;
    uint32_t eqb[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      eqb[i] = eq_before;
      const uint32_t left = quota > eq_before ? quota - eq_before : 0u;
      ws[i] = e < n ? ctl.warp_mass[e] + min(left, eqs[i]) * w_end : 0ull;
      run += ws[i];
      eq_before += eqs[i];
    }
    unsigned long long in = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long y = shfl_up64(in, d);
      if (lane >= d) in += y;
    }
    const unsigned long long total = __shfl_sync(0xffffffffu, in, 31);
    const float u = fminf(fmaxf(a.u[t], 0.0f), 0x1.fffffep-1f);
    const unsigned long long target = __umul64hi(static_cast<unsigned long long>(static_cast<double>(u) * 0x1p64), total);
    unsigned long long before = in - run;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      if (e < n && before <= target && target < before + ws[i] && e / kWarps == R) {
        ctl.hit_warp = e % kWarps;
        ctl.hit_eq = eqb[i];
        ctl.hit_before = before;
        ctl.total = total;
        ctl.target = target;
      }
      before += ws[i];
    }
  }
  __syncthreads();
  if (warp != ctl.hit_warp) return;

  // ---- its run in order: 32 pieces at a time
  const unsigned long long target = ctl.target, total = ctl.total;
  unsigned long long before = ctl.hit_before;
  uint32_t eq_before = ctl.hit_eq;
  for (int i0 = warp * chunk; i0 < (warp + 1) * chunk; i0 += 32) {
    const int i = i0 + lane;
    uint4 v = make_uint4(kNone, kNone, kNone, kNone);
    if (i < (warp + 1) * chunk) v = seg[i];
    uint32_t n_eq = 0;
#pragma unroll
    for (int m = 0; m < VE; ++m) n_eq += key_of(element<BF16>(v, m)) == kept.key && i < (warp + 1) * chunk;
    uint32_t eq_in = n_eq;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, eq_in, d);
      if (lane >= d) eq_in += y;
    }
    auto kept_weight = [&](float x, uint32_t& rank) -> unsigned long long {
      const uint32_t key = key_of(x);
      if (key > kept.key) {
        const unsigned long long w = r.weight(x);
        return w >= least ? w : 0ull;
      }
      return key == kept.key && rank++ < quota ? w_end : 0ull;
    };
    unsigned long long run = 0;
    uint32_t rank = eq_before + eq_in - n_eq;
    if (i < (warp + 1) * chunk) {
#pragma unroll
      for (int m = 0; m < VE; ++m) run += kept_weight(element<BF16>(v, m), rank);
    }
    unsigned long long in = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long y = shfl_up64(in, d);
      if (lane >= d) in += y;
    }
    const unsigned long long mine = before + in - run;
    const bool hit = mine <= target && target < mine + run;
    if (hit) {
      unsigned long long at = mine;
      rank = eq_before + eq_in - n_eq;
#pragma unroll
      for (int m = 0; m < VE; ++m) {
        const float x = element<BF16>(v, m);
        const unsigned long long w = kept_weight(x, rank);
        if (at <= target && target < at + w) {
          a.tokens[t] = (v0 + i) * VE + m - mis;
          if (a.logp) {
            // by the difference where the token has most of the weight, else by the logit
            if (w > total / 4) a.logp[t] = -log1pf(static_cast<float>(total - w) / static_cast<float>(w));
            else a.logp[t] = (x - mx) * (r.c_hi * 0.69314718f) - logf(static_cast<float>(total) * 0x1p-43f);
          }
        }
        at += w;
      }
    }
    if (__any_sync(0xffffffffu, hit)) return;
    before += __shfl_sync(0xffffffffu, in, 31);
    eq_before += __shfl_sync(0xffffffffu, eq_in, 31);
  }
}

// CTAs of a row: a power of two, so that a CTA has some 64 KB of it at most.
int cluster_of(int V, bool bf16) {
  const int64_t bytes = static_cast<int64_t>(V) * (bf16 ? 2 : 4);
  int C = 1;
  while (C < kMaxCluster && bytes > static_cast<int64_t>(C) * 16384) C *= 2;
  return C;
}

struct Plan {
  int C, chunk;
  size_t smem;
};
Plan plan_of(int V, bool bf16) {
  const int VE = bf16 ? 8 : 4;
  Plan p;
  p.C = cluster_of(V, bf16);
  const int64_t vecs = (static_cast<int64_t>(V) + 2 * (VE - 1)) / VE + 1;  // wherever the row starts
  p.chunk = static_cast<int>((vecs + p.C * kWarps - 1) / (p.C * kWarps));
  p.smem = static_cast<size_t>(p.chunk) * kWarps * 16 + sizeof(Control) + static_cast<size_t>(kBins / p.C) * 2 * 12;
  return p;
}

}  // namespace

// what eight CTAs' shared memory holds
bool sample_supported(int V, bool bf16) { return V <= (bf16 ? 800000 : 400000) && plan_of(V, bf16).smem <= 227 * 1024; }

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  const Plan p = plan_of(a.V, a.bf16 != 0);
  void (*kernel)(SampleArgs, int) = a.bf16 ? k_sample<true> : k_sample<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T) * p.C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, p.chunk);
}

}  // namespace mxk
