// A token from a row of logits by temperature, top-k, top-p and min-p and one given
// random number, by the inverse of the distribution function in the order of the
// tokens' numbers.
//
// A cluster of CTAs holds the row in its shared memory (read once) and goes over it a
// few times from there:
//   1. the row's maximum m;
//   2. with top-k or top-p, a histogram of counts (and weights) over bins of m - logit,
//      merged across the cluster slice by slice, which tells the bin where the kept prefix
//      ends.  As a rule the tokens up to there are few: one CTA gathers them and does the
//      rest alone, by radix selections over what its threads hold in registers;
//   3. where they are many, the end is found in its bin alone (by a CTA if that is small,
//      else by further histograms over the bits of the logit); then the kept weights are
//      added up by warp, and the warp in which the random number falls goes over its
//      stretch once more.  So are rows without top-k and top-p.
//
// Weights are whole numbers, 2^43 e^((logit - m) / temperature) rounded down, so sums
// are exact in any order (no atomic changes a result) and two calls agree.  A draw next
// to a token's border is decided by the weights' own rounding: e^x is taken in two floats
// with a table of 2^(j/64), 2^-31 off where one float's exponential would be 2^-22, as a
// vocabulary has 10^5 borders (table-driven reduction, P. T. P. Tang 1989, and the Taylor series
// of 2^f).  Weights below 2^-43 of the largest are zero.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <climits>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace mxk {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kDigit = 10;  // bins of a histogram, bits of the logit that one divides by
constexpr int kItems = 3;                 // tokens that a thread holds of those gathered in one CTA
constexpr int kCandidates = 1280;         // most of those: their list lies where the histogram was
constexpr int kMaxCluster = 8;
constexpr int kOneBits = 43;
constexpr unsigned long long kOne = 1ull << kOneBits;  // the largest weight; 2^20 of them fit 64 bits

// 2^(j/64): 2^43 times it as a whole number (low word, high word), and as a float's bits.
__constant__ uint4 kExp2[64] = {
    {0x0u, 0x800u, 0x3f800000u, 0u}, {0x4d1f3bc0u, 0x816u, 0x3f8164d2u, 0u},
    {0xd8698ac3u, 0x82cu, 0x3f82cd87u, 0u}, {0xa28c3aceu, 0x843u, 0x3f843a29u, 0u},
    {0xac367cc5u, 0x85au, 0x3f85aac3u, 0u}, {0xf61969e9u, 0x871u, 0x3f871f62u, 0u},
    {0x80e8092eu, 0x889u, 0x3f88980fu, 0u}, {0x4d575497u, 0x8a1u, 0x3f8a14d5u, 0u},
    {0x5c1e3ea9u, 0x8b9u, 0x3f8b95c2u, 0u}, {0xadf5b7e6u, 0x8d1u, 0x3f8d1adfu, 0u},
    {0x4398b45du, 0x8eau, 0x3f8ea43au, 0u}, {0x1dc43146u, 0x903u, 0x3f9031dcu, 0u},
    {0x3d373ab1u, 0x91cu, 0x3f91c3d3u, 0u}, {0xa2b2f13eu, 0x935u, 0x3f935a2bu, 0u},
    {0x4efa8fefu, 0x94fu, 0x3f94f4f0u, 0u}, {0x42d37202u, 0x969u, 0x3f96942du, 0u},
    {0x7f0518dcu, 0x983u, 0x3f9837f0u, 0u}, {0x459320bu, 0x99eu, 0x3f99e046u, 0u},
    {0xd39b9d55u, 0x9b8u, 0x3f9b8d3au, 0u}, {0xed9a72d0u, 0x9d3u, 0x3f9d3edau, 0u},
    {0x5326091au, 0x9efu, 0x3f9ef532u, 0u}, {0x510fb97u, 0xa0bu, 0x3fa0b051u, 0u},
    {0x43030c5u, 0xa27u, 0x3fa27043u, 0u}, {0x515ae09eu, 0xa43u, 0x3fa43516u, 0u},
    {0xed6a9b15u, 0xa5fu, 0x3fa5fed7u, 0u}, {0xd93b4e96u, 0xa7cu, 0x3fa7cd94u, 0u},
    {0x15ab4ea8u, 0xa9au, 0x3fa9a15bu, 0u}, {0xa39b5a94u, 0xab7u, 0x3fab7a3au, 0u},
    {0x83eea42au, 0xad5u, 0x3fad583fu, 0u}, {0xb78ad691u, 0xaf3u, 0x3faf3b79u, 0u},
    {0x3f581d2bu, 0xb12u, 0x3fb123f6u, 0u}, {0x1c412a91u, 0xb31u, 0x3fb311c4u, 0u},
    {0x4f333f9eu, 0xb50u, 0x3fb504f3u, 0u}, {0xd91e328du, 0xb6fu, 0x3fb6fd92u, 0u},
    {0xbaf47630u, 0xb8fu, 0x3fb8fbafu, 0u}, {0xf5ab2134u, 0xbafu, 0x3fbaff5bu, 0u},
    {0x8a39f581u, 0xbd0u, 0x3fbd08a4u, 0u}, {0x799b67a7u, 0xbf1u, 0x3fbf179au, 0u},
    {0xc4cca667u, 0xc12u, 0x3fc12c4du, 0u}, {0x6ccda249u, 0xc34u, 0x3fc346cdu, 0u},
    {0x72a11550u, 0xc56u, 0x3fc5672au, 0u}, {0xd74c8abcu, 0xc78u, 0x3fc78d75u, 0u},
    {0x9bd866e3u, 0xc9bu, 0x3fc9b9beu, 0u}, {0xc14fef27u, 0xcbeu, 0x3fcbec15u, 0u},
    {0x48c151f8u, 0xce2u, 0x3fce248cu, 0u}, {0x333daef3u, 0xd06u, 0x3fd06334u, 0u},
    {0x81d91f13u, 0xd2au, 0x3fd2a81eu, 0u}, {0x35aabcffu, 0xd4fu, 0x3fd4f35bu, 0u},
    {0x4fccad6au, 0xd74u, 0x3fd744fdu, 0u}, {0xd15c278bu, 0xd99u, 0x3fd99d16u, 0u},
    {0xbb797dafu, 0xdbfu, 0x3fdbfbb8u, 0u}, {0xf4825e1u, 0xde6u, 0x3fde60f5u, 0u},
    {0xcdeec2a9u, 0xe0cu, 0x3fe0ccdfu, 0u}, {0xf8972be9u, 0xe33u, 0x3fe33f89u, 0u},
    {0x906e77c8u, 0xe5bu, 0x3fe5b907u, 0u}, {0x96a503c5u, 0xe83u, 0x3fe8396au, 0u},
    {0xc6e7dd2u, 0xeacu, 0x3feac0c7u, 0u}, {0xf301ed99u, 0xed4u, 0x3fed4f30u, 0u},
    {0x4b99bdceu, 0xefeu, 0x3fefe4bau, 0u}, {0x1773c5a0u, 0xf28u, 0x3ff28177u, 0u},
    {0x57d15248u, 0xf52u, 0x3ff5257du, 0u}, {0xdf730adu, 0xf7du, 0x3ff7d0dfu, 0u},
    {0x3b2db723u, 0xfa8u, 0x3ffa83b3u, 0u}, {0xe0c0cf48u, 0xfd3u, 0x3ffd3e0cu, 0u},
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

// Where a selection ends: items above `key`, and some of the `count` with it.
struct Selected {
  uint32_t key, before, count;
  unsigned long long before_mass;
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
  uint32_t n;  // candidates (rank 0)
  uint32_t local_n, local_base, local_at[kCandidates];  // this CTA's
  uint32_t gathered[kMaxCluster];
  Selected sel;
  uint32_t sel_digit;
  uint32_t sel_count[256], sel_lo[256], sel_hi[256];
  uint32_t rank_n;
  unsigned long long rank_order[128], rank_w[128], near_before, near_order;
  int near_bin;
  uint32_t warp_eq[kMaxCluster * kWarps];
  unsigned long long warp_mass[kMaxCluster * kWarps];
  int hit_warp;
  uint32_t hit_eq;
  unsigned long long hit_before, total, target;
  uint32_t red[kWarps], red2[kWarps];
  unsigned long long red64[kWarps];
  uint4 exp2_table[64];
  union {
    struct {
      uint32_t hist_count[kBins], hist_lo[kBins], hist_hi[kBins];
    };
    struct {
      uint32_t cand_key[kCandidates], cand_at[kCandidates];  // (rank 0) behind the histogram's merge
    };
  };
};
static_assert(kCandidates <= kItems * kThreads && 2 * kCandidates <= 3 * kBins, "");

// Logits in their order as unsigned numbers (both zeros the same), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// x in (0, 1] times 2^bits as a whole number, rounded down, without the slow 64-bit floats
// (24-bit significands: nothing is lost above 2^-40).
__device__ __forceinline__ unsigned long long fixed_of(float x, int bits) {
  if (!(x > 0.0f)) return 0ull;
  const uint32_t b = __float_as_uint(x);
  const int e = max(static_cast<int>(b >> 23), 1);  // subnormals give 0 below
  const unsigned long long m = (b & 0x7FFFFFu) | (b >> 23 ? 0x800000u : 0u);
  const int up = bits + e - 150;
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0ull;
}

// mx = max(mx, the piece's elements), NaN where one is.
template <bool BF16>
__device__ __forceinline__ void piece_max(const uint4& v, float& mx) {
  if (BF16) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(a << 16)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(a & 0xFFFF0000u)));
  } else {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(v.x)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(v.y)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(v.z)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(mx) : "f"(__uint_as_float(v.w)));
  }
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
  float max, least;   // the row's largest logit; the least one with a weight
  float c_hi, c_lo;   // log2(e) / temperature
  float bin_scale;
  uint32_t table;     // shared-memory address of kExp2
  // 2^43 e^((x - max) / temperature), rounded down.  Without branches, so that a thread's
  // weights go side by side.
  __device__ __forceinline__ unsigned long long weight(float x) const {
    if (max == INFINITY) return x == max ? kOne : 0ull;
    const bool none = x < least;  // -inf among them
    x = fmaxf(x, least);
    const float s = x - max;
    const float t = s * c_hi;
    float t_lo = fmaf(s, c_lo, fmaf(s, c_hi, -t));
    if (!BF16) {
      // x - max = s + e exactly (the error of a sum of two floats); of 8-bit significands s is
      // exact, but for logits below 2^-16 of the largest (there 2^-22 of a weight)
      const float v = s - x;
      t_lo = fmaf((x - (s - v)) - (max + v), c_hi, t_lo);
    }
    const float shifted = t + 196608.0f;  // 1.5 * 2^17: the sum's last place is 2^-6, its last bits t's
    const uint32_t bits = __float_as_uint(shifted);
    const float f = (t - (shifted - 196608.0f)) + t_lo;
    // 2^36 (2^f - 1) for |f| <= 2^-7: the next term is below 2^-44 of the weight
    const float q = f * fmaf(f, fmaf(f, fmaf(f, 9.6181291e-3f * 0x1p36f, 5.5504109e-2f * 0x1p36f), 0.24022651f * 0x1p36f), 0.69314718f * 0x1p36f);
    uint32_t lo, hi, p, unused;
    asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(lo), "=r"(hi), "=r"(p), "=r"(unused) : "r"(table + (bits & 63u) * 16u));
    const unsigned long long whole = static_cast<unsigned long long>(hi) << 32 | lo;
    const long long part = static_cast<long long>(__float2int_rn(__uint_as_float(p) * q)) * (1 << (kOneBits - 36));  // below 2^-6 in size
    const unsigned long long w = (whole + part) >> ((0x4840003Fu - bits) >> 6);
    return none ? 0ull : w;
  }
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

__device__ __forceinline__ void histogram_begin(Control& ctl) {
  for (int b = threadIdx.x; b < kBins; b += kThreads) ctl.hist_count[b] = ctl.hist_lo[b] = ctl.hist_hi[b] = 0u;
  __syncthreads();
}

// The CTAs' histograms merged in slices of kBins / C bins, one a CTA, and the slices' sums
// known to all.
__device__ void histogram_merge(Control& ctl, uint32_t* slice_count, unsigned long long* slice_mass, bool masses, int level) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  cluster.sync();
  const int S = kBins / C;
  uint32_t count = 0;
  unsigned long long mass = 0;
  for (int b = tid; b < S; b += kThreads) {
    // all peers' bins are on their way before the first is added
    const int at = R * S + b;
    uint32_t ns[kMaxCluster], lo[kMaxCluster], hi[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      ns[c] = lo[c] = hi[c] = 0u;
      if (c < C) {
        const Control* peer = cluster.map_shared_rank(&ctl, c);
        ns[c] = peer->hist_count[at];
        if (masses) {
          lo[c] = peer->hist_lo[at];
          hi[c] = peer->hist_hi[at];
        }
      }
    }
    uint32_t n = 0;
    unsigned long long w = 0;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      n += ns[c];
      w += (static_cast<unsigned long long>(hi[c]) << 32) + lo[c];
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

// Histogram of the whole row (level 0) or of a subset by the `kDigit` bits below its
// shift, highest first; merged.
template <bool BF16>
__device__ void histogram(const Row<BF16>& r, Control& ctl, uint32_t* slice_count, unsigned long long* slice_mass, bool masses,
                          int level, const Subset& sub) {
  const int tid = threadIdx.x, lane = tid & 31;
  histogram_begin(ctl);
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
    unsigned long long w[Row<BF16>::VE];
#pragma unroll
    for (int m = 0; m < Row<BF16>::VE; ++m) w[m] = masses ? r.weight(element<BF16>(v, m)) : 0ull;
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
      if (b == kBins - 1) {
        ++last_count;
        last_mass += w[m];
      } else {
        atomicAdd(&ctl.hist_count[b], 1u);
        if (w[m]) add(b, w[m]);
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
  histogram_merge(ctl, slice_count, slice_mass, masses, level);
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

// Tokens gathered in one CTA, up to kItems a thread.
struct Items {
  uint32_t key[kItems], at[kItems];
  unsigned long long w[kItems];
  uint32_t kept;  // bit i: item i is there and still kept
};

// Sum over the CTA, the same in every thread.
__device__ unsigned long long block_sum(Control& ctl, unsigned long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();  // the slots may still be read from the call before
  if ((threadIdx.x & 31) == 0) ctl.red64[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += ctl.red64[i];
  return v;
}

// The key, in descending order, at which the `target`th of the kept items, or unit of their
// weight, lies, beginning behind `before` items of `before_mass` (the weight before it is
// told with `masses`).  Whole CTA.
__device__ Selected select(Control& ctl, const uint32_t (&key)[kItems], const unsigned long long (&w)[kItems], uint32_t kept, bool by_mass, bool masses,
                           unsigned long long target, uint32_t before, unsigned long long before_mass) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (kept >> i & 1) {
      lo = min(lo, key[i]);
      hi = max(hi, key[i]);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t mine = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(__popc(kept)));
  __syncthreads();
  if (lane == 0) {
    ctl.red[warp] = lo;
    ctl.red2[warp] = hi;
    ctl.red64[warp] = mine;
  }
  __syncthreads();
  Selected r{0u, before, 0u, before_mass};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    lo = min(lo, ctl.red[i]);
    hi = max(hi, ctl.red2[i]);
    r.count += static_cast<uint32_t>(ctl.red64[i]);
  }
  r.key = hi;
  if (lo >= hi) return r;  // all the same
  int shift = 32 - __clz(lo ^ hi);
  uint32_t prefix = shift < 32 ? hi >> shift : 0u;
  while (shift > 0 && r.count > 1) {
    const int low = max(shift - 8, 0), bits = shift - low;
    for (int i = tid; i < 256; i += kThreads) ctl.sel_count[i] = ctl.sel_lo[i] = ctl.sel_hi[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if ((kept >> i & 1) && (shift >= 32 || (key[i] >> shift) == prefix)) {
        const uint32_t d = (key[i] >> low) & ((1u << bits) - 1);
        atomicAdd(&ctl.sel_count[d], 1u);
        if (masses) {
          const uint32_t l = static_cast<uint32_t>(w[i]);
          const uint32_t h = static_cast<uint32_t>(w[i] >> 32) + (atomicAdd(&ctl.sel_lo[d], l) > ~l ? 1u : 0u);
          if (h) atomicAdd(&ctl.sel_hi[d], h);
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8 l and the seven below
      uint32_t n[8], run = 0;
      unsigned long long m[8], run_mass = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = 255 - 8 * lane - i;
        n[i] = ctl.sel_count[d];
        m[i] = (static_cast<unsigned long long>(ctl.sel_hi[d]) << 32) + ctl.sel_lo[d];
        run += n[i];
        run_mass += m[i];
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
      const bool reached = by_mass ? r.before_mass + in_mass >= target : r.before + in >= target;
      const unsigned hits = __ballot_sync(0xffffffffu, reached);
      if (lane == (hits ? __ffs(hits) - 1 : 31)) {
        uint32_t b = r.before + in - run;
        unsigned long long bm = r.before_mass + in_mass - run_mass;
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!found) {
            if ((by_mass ? bm + m[i] : static_cast<unsigned long long>(b + n[i])) >= target || i == 7) {
              ctl.sel = Selected{0u, b, n[i], bm};
              ctl.sel_digit = 255 - 8 * lane - i;
              found = true;
            } else {
              b += n[i];
              bm += m[i];
            }
          }
        }
      }
    }
    __syncthreads();
    r = ctl.sel;
    prefix = prefix << bits | ctl.sel_digit;
    shift = low;
  }
  // the one item, or the equal ones, left
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if ((kept >> i & 1) && (shift >= 32 || (key[i] >> shift) == prefix)) ctl.sel.key = key[i];
  __syncthreads();
  r.key = ctl.sel.key;
  return r;
}

// The same by 1024 even bins of the items' range, and the few items of one bin ranked one
// against the other: one pass where the radix selection takes one for each eight bits.
// Items are in ascending `order`; the order of the item at which the target lies.  Whole CTA.
constexpr int kRanked = 128;  // most items of that bin
__device__ unsigned long long select_near(Control& ctl, const int (&bin)[kItems], const unsigned long long (&order)[kItems],
                                          const unsigned long long (&w)[kItems], uint32_t kept, bool by_mass, unsigned long long target, bool& done) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kNear = 2 * kThreads;
  static_assert(kNear == kBins, "the bins lie where the histogram and the list were");
  __syncthreads();
  for (int i = tid; i < kNear; i += kThreads) ctl.hist_count[i] = ctl.hist_lo[i] = ctl.hist_hi[i] = 0u;
  if (tid == 0) {
    ctl.rank_n = 0u;
    ctl.near_bin = 0;  // a bin, also where no bin reaches the target
    ctl.near_before = 0ull;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (kept >> i & 1) {
      atomicAdd(&ctl.hist_count[bin[i]], 1u);
      if (by_mass) {
        const uint32_t l = static_cast<uint32_t>(w[i]);
        const uint32_t h = static_cast<uint32_t>(w[i] >> 32) + (atomicAdd(&ctl.hist_lo[bin[i]], l) > ~l ? 1u : 0u);
        if (h) atomicAdd(&ctl.hist_hi[bin[i]], h);
      }
    }
  }
  __syncthreads();
  // each thread two bins; what lies before them by warp and then over the warps
  const unsigned long long v0 = by_mass ? (static_cast<unsigned long long>(ctl.hist_hi[2 * tid]) << 32) + ctl.hist_lo[2 * tid] : ctl.hist_count[2 * tid];
  const unsigned long long v1 = by_mass ? (static_cast<unsigned long long>(ctl.hist_hi[2 * tid + 1]) << 32) + ctl.hist_lo[2 * tid + 1] : ctl.hist_count[2 * tid + 1];
  unsigned long long in = v0 + v1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long y = shfl_up64(in, d);
    if (lane >= d) in += y;
  }
  if (lane == 31) ctl.red64[warp] = in;
  __syncthreads();
  unsigned long long before = in - v0 - v1;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) before += i < warp ? ctl.red64[i] : 0ull;
  if (before < target && before + v0 + v1 >= target) {
    const int second = before + v0 < target;
    ctl.near_bin = 2 * tid + second;
    ctl.near_before = second ? before + v0 : before;
  }
  __syncthreads();
  const int b = ctl.near_bin;
  done = ctl.hist_count[b] <= kRanked;
  if (!done) return 0ull;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if ((kept >> i & 1) && bin[i] == b) {
      const uint32_t at = atomicAdd(&ctl.rank_n, 1u);
      ctl.rank_order[at] = order[i];
      ctl.rank_w[at] = by_mass ? w[i] : 1ull;
    }
  }
  __syncthreads();
  const int n = static_cast<int>(ctl.rank_n);
  if (tid < n) {
    const unsigned long long mine = ctl.rank_order[tid], own = ctl.rank_w[tid];
    unsigned long long sum = ctl.near_before;
    for (int j = 0; j < n; ++j) sum += ctl.rank_order[j] < mine ? ctl.rank_w[j] : 0ull;
    if (sum < target && sum + own >= target) ctl.near_order = mine;
  }
  __syncthreads();
  return ctl.near_order;
}

// Keeps of the items the prefix, by logit and then number, of `target` items, or until
// their weight reaches target.
template <bool BF16>
__device__ void keep_prefix(const Row<BF16>& r, Control& ctl, Items& it, float near_scale, bool by_mass, unsigned long long target) {
  int bin[kItems];
  unsigned long long order[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const float x = value_of(it.key[i]);
    bin[i] = x == r.max ? 0 : min(2 * kThreads - 1, __float2int_rz((r.max - x) * near_scale));
    order[i] = static_cast<unsigned long long>(~it.key[i]) << 32 | it.at[i];
  }
  bool done;
  const unsigned long long last = select_near(ctl, bin, order, it.w, it.kept, by_mass, target, done);
  if (done) {
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (order[i] > last) it.kept &= ~(1u << i);
    return;
  }
  const Selected s = select(ctl, it.key, it.w, it.kept, by_mass, by_mass, target, 0u, 0ull);
  uint32_t equal = 0, above = 0;
  unsigned long long w = 0;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (it.kept >> i & 1) {
      if (it.key[i] > s.key) above |= 1u << i;
      if (it.key[i] == s.key) {
        equal |= 1u << i;
        w = it.w[i];
      }
    }
  }
  if (s.count > 1) {
    // of equal ones the first by number
    if (by_mass) {
      __syncthreads();
      if (equal) ctl.total = w;
      __syncthreads();
      w = ctl.total;
    }
    unsigned long long quota = by_mass ? (w ? (target - s.before_mass + w - 1) / w : s.count) : target - s.before;
    if (quota < s.count) {
      uint32_t at[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) at[i] = ~it.at[i];
      const Selected last = select(ctl, at, it.w, equal, false, false, quota, 0u, 0ull);
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (at[i] < last.key) equal &= ~(1u << i);
    }
  }
  it.kept = above | equal;
}

// The tokens of bins up to sub.bin0 (all_before), or of a subset, into rank 0's list: first
// into one of this CTA's, then all of them with one reservation.  Whole CTA; the CTAs'
// numbers of them are in `gathered` behind the next cluster barrier (more than kCandidates
// in all: the list does not hold them).
template <bool BF16>
__device__ void gather(const Row<BF16>& r, Control& ctl, const Subset& sub, bool all_before) {
  const int tid = threadIdx.x;
  if (tid == 0) ctl.local_n = 0u;
  __syncthreads();
  // some more than the bins' tokens do no harm: the list is ranked exactly
  const float edge = sub.bin0 >= kBins - 1 ? -INFINITY : r.max - static_cast<float>(sub.bin0 + 1) / r.bin_scale * 1.00001f;
  auto take = [&](int at) {
    const uint32_t n = atomicAdd(&ctl.local_n, 1u);
    if (n < kCandidates) ctl.local_at[n] = static_cast<uint32_t>(at);
  };
  for (int i = tid; i < r.vecs; i += kThreads) {
    const uint4 v = r.seg[i];
    if (all_before) {
      float top = -INFINITY;
      piece_max<BF16>(v, top);
      if (!(top >= edge)) continue;
    }
#pragma unroll
    for (int m = 0; m < Row<BF16>::VE; ++m) {
      const float x = element<BF16>(v, m);
      if (all_before ? x >= edge : sub.holds(r, x, key_of(x))) take(i * Row<BF16>::VE + m);
    }
  }
  __syncthreads();
  cg::cluster_group cluster = cg::this_cluster();
  Control* leader = cluster.map_shared_rank(&ctl, 0);
  if (tid == 0) ctl.local_base = atomicAdd(&leader->n, ctl.local_n);
  if (tid < static_cast<int>(cluster.num_blocks())) cluster.map_shared_rank(&ctl, tid)->gathered[cluster.block_rank()] = ctl.local_n;
  __syncthreads();
  const uint32_t base = ctl.local_base;
  for (uint32_t i = tid; i < min(ctl.local_n, static_cast<uint32_t>(kCandidates)); i += kThreads) {
    if (base + i < kCandidates) {
      const uint32_t at = ctl.local_at[i];
      const uint32_t word = reinterpret_cast<const uint32_t*>(r.seg)[BF16 ? at / 2 : at];
      const float x = __uint_as_float(!BF16 ? word : at & 1 ? word & 0xFFFF0000u : word << 16);
      leader->cand_key[base + i] = key_of(x);
      leader->cand_at[base + i] = r.at0 + at;
    }
  }
}

template <bool BF16>
__device__ Items take_items(const Row<BF16>& r, const Control& ctl, uint32_t n) {
  Items it;
  it.kept = 0;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const uint32_t at = threadIdx.x + i * kThreads;
    it.key[i] = it.at[i] = 0u;
    it.w[i] = 0ull;
    if (at < n) {
      it.key[i] = ctl.cand_key[at];
      it.at[i] = ctl.cand_at[at];
      it.w[i] = r.weight(value_of(it.key[i]));
      it.kept |= 1u << i;
    }
  }
  return it;
}

// Where the prefix of `target` tokens (or of tokens until their weights reach target)
// ends, from its bin `f` of the level-0 histogram on.
template <bool BF16>
__device__ End find_end(const Row<BF16>& r, Control& ctl, uint32_t* const (&slice_count)[2], unsigned long long* const (&slice_mass)[2],
                        bool by_mass, bool masses, unsigned long long target, Found f) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  Subset sub{f.bin, 32, 0u};
  while (f.count > kCandidates && sub.shift > (BF16 ? 16 : 0)) {  // by the next bits of the logit
    histogram(r, ctl, slice_count[1], slice_mass[1], masses, 1, sub);
    const Found next = find_bin(ctl, slice_count[1], slice_mass[1], by_mass, target, 1, f);
    const int low = sub.shift - kDigit, digit = kBins - 1 - next.bin;
    sub.prefix = sub.shift >= 32 ? digit : low >= 0 ? (sub.prefix << kDigit) | digit : (sub.prefix << sub.shift) | (digit >> -low);
    sub.shift = max(low, 0);
    f = next;
  }
  if (f.count > kCandidates) {
    // all bits are known: equal logits, the first ones by number (of bf16 the last bits are 0, but for
    // the sign's complement)
    uint32_t key = sub.prefix << sub.shift;
    if (BF16 && !(key & 0x80000000u)) key |= 0xFFFFu;
    const unsigned long long w = masses ? r.weight(value_of(key)) : 0ull;
    unsigned long long quota = by_mass ? (w ? (target - f.before_mass + w - 1) / w : f.count) : target - f.before;
    if (quota > f.count) quota = f.count;
    return End{key, static_cast<uint32_t>(quota), f.before_mass + quota * w};
  }
  gather(r, ctl, sub, false);
  cluster.sync();
  if (R == 0) {
    const Items it = take_items(r, ctl, f.count);
    const Selected s = select(ctl, it.key, it.w, it.kept, by_mass, masses, target, f.before, f.before_mass);
    if (threadIdx.x == 0) {
      const unsigned long long w = masses ? r.weight(value_of(s.key)) : 0ull;
      unsigned long long quota = by_mass ? (w ? (target - s.before_mass + w - 1) / w : s.count) : target - s.before;
      if (quota > s.count) quota = s.count;
      const End e{s.key, static_cast<uint32_t>(quota), s.before_mass + quota * w};
      for (int c = 0; c < C; ++c) cluster.map_shared_rank(&ctl, c)->end = e;
    }
  }
  cluster.sync();
  return ctl.end;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleArgs a, int chunk) {
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int VE = Row<BF16>::VE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), R = cluster.block_rank();
  const int t = blockIdx.x / C;
  cluster_arrive_relaxed();  // waited for ahead of the first store to a peer, which has to have started by then
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
  float mx = -INFINITY;  // NaN as soon as one is seen
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
      piece_max<BF16>(v[u], mx);
    }
  }
  if (tid < 64) ctl.exp2_table[tid] = kExp2[tid];
  if (tid == 0) {
    const double c = 1.4426950408889634074 / static_cast<double>(fminf(fmaxf(temperature, 0x1p-126f), 0x1p100f));  // finite as a float
    ctl.c_hi = static_cast<float>(c);
    ctl.c_lo = static_cast<float>(c - static_cast<double>(ctl.c_hi));
  }
  const int any_nan = __syncthreads_or(mx != mx);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  if (lane == 0) ctl.red[warp] = __float_as_uint(mx);
  __syncthreads();
  cluster_wait();
  if (tid < C) {
    for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, __uint_as_float(ctl.red[i]));
    Control* peer = cluster.map_shared_rank(&ctl, tid);
    peer->max[R] = mx;
    peer->nan[R] = any_nan;
  }
  cluster.sync();
  bool bad = !(temperature >= 0.0f) || isnan(top_p) || isnan(min_p);
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
  r.table = smem_u32(ctl.exp2_table);
  r.least = fmaxf(mx - 45.0f / r.c_hi, -3.402823466e38f);
  // the first histogram spans what has weight (e^-30), and eight units of the logits at least
  r.bin_scale = kBins / fmaxf(30.0f * 1.4426950f / r.c_hi, 8.0f);

  const unsigned long long least = fixed_of(fminf(min_p, 1.0f), kOneBits);
  const float u = fminf(fmaxf(a.u[t], 0.0f), 0x1.fffffep-1f);
  const unsigned long long u64 = fixed_of(u, 64);
  auto log_share = [&](float x, unsigned long long w, unsigned long long total) {
    // by the difference where the token has most of the weight, else by the logit
    if (w > total / 4) return -log1pf(static_cast<float>(total - w) / static_cast<float>(w));
    const float below = mx == INFINITY ? 0.0f : x - mx;  // of infinite logits only those of the maximum have a weight
    return below * (r.c_hi * 0.69314718f) - logf(static_cast<float>(total) * 0x1p-43f);
  };

  // ---- the kept prefix
  const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.0f;
  // a token is kept while the weight before it is below p times the whole: the whole
  // numbers below that product are those below its ceiling
  const unsigned long long p64 = by_p ? fixed_of(top_p, 64) : 0ull;
  auto p_target = [&](unsigned long long mass) {
    const unsigned long long target = __umul64hi(p64, mass) + (p64 * mass ? 1ull : 0ull);
    return target ? target : 1ull;
  };
  End kept{0u, UINT_MAX, 0ull};
  if (by_k || by_p) {
    unsigned long long target = static_cast<unsigned long long>(top_k);
    // With a small top-k: where so many of the pieces' maxima lie, so many tokens do, and few
    // others, so the histogram is one of maxima, an addition for four or eight tokens, without
    // weights.
    const bool maxima = by_k && top_k <= kCandidates * 7 / 8 && top_k <= a.V / (2 * VE);
    bool masses = by_p && !maxima;
    Found f;
    if (maxima) {
      histogram_begin(ctl);
      for (int i = tid; i < per; i += kThreads) {
        float top = -INFINITY;
        piece_max<BF16>(seg[i], top);
        const int b = r.bin(top);
        if (b < kBins - 1) atomicAdd(&ctl.hist_count[b], 1u);  // (the last bin's are found missing below)
      }
      histogram_merge(ctl, slice_count[0], slice_mass[0], false, 0);
      f = find_bin(ctl, slice_count[0], slice_mass[0], false, target, 0, Found{});
    } else {
      histogram(r, ctl, slice_count[0], slice_mass[0], masses, 0, Subset{0, 32, 0u});
      if (!by_k) {
        unsigned long long mass = 0;
        for (int c = 0; c < C; ++c) mass += ctl.slice_mass[0][c];
        target = p_target(mass);
      }
      f = find_bin(ctl, slice_count[0], slice_mass[0], !by_k, target, 0, Found{});
    }
    if (maxima || f.before + f.count <= kCandidates) {
      // ---- few tokens: one CTA does the rest
      gather(r, ctl, Subset{f.bin, 32, 0u}, true);
      cluster.sync();
      uint32_t n = 0;
      for (int c = 0; c < C; ++c) n += ctl.gathered[c];
      if (n <= kCandidates && n >= static_cast<uint32_t>(by_k ? top_k : 1)) {
        if (R != 0) return;  // from here on no CTA touches another's memory
        const float near_scale = r.bin_scale * (2 * kThreads) / static_cast<float>(f.bin + 1);
        Items it = take_items(r, ctl, n);
        keep_prefix(r, ctl, it, near_scale, !by_k, target);
        if (by_k && by_p) {
          unsigned long long mass = 0;
#pragma unroll
          for (int i = 0; i < kItems; ++i) mass += it.kept >> i & 1 ? it.w[i] : 0ull;
          keep_prefix(r, ctl, it, near_scale, true, p_target(block_sum(ctl, mass)));
        }
        unsigned long long mass = 0, order[kItems];
        int bin[kItems];
        const float places = (2 * kThreads) / (static_cast<float>(a.V) + 16.0f);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          if (it.w[i] < least) it.kept &= ~(1u << i);
          mass += it.kept >> i & 1 ? it.w[i] : 0ull;
          order[i] = it.at[i];
          bin[i] = min(2 * kThreads - 1, __float2int_rz(static_cast<float>(it.at[i]) * places));
        }
        const unsigned long long total = block_sum(ctl, mass), draw = __umul64hi(u64, total) + 1;
        bool done;
        unsigned long long drawn = select_near(ctl, bin, order, it.w, it.kept, true, draw, done);
        if (!done) {
          uint32_t at[kItems];
#pragma unroll
          for (int i = 0; i < kItems; ++i) at[i] = ~it.at[i];
          drawn = ~select(ctl, at, it.w, it.kept, true, true, draw, 0u, 0ull).key;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          if ((it.kept >> i & 1) && it.at[i] == static_cast<uint32_t>(drawn)) {
            a.tokens[t] = static_cast<int32_t>(it.at[i]) - mis;
            if (a.logp) a.logp[t] = log_share(value_of(it.key[i]), it.w[i], total);
          }
        }
        return;
      }
      // More of them than the list holds: some lie on the border behind the prefix's bin (or, of
      // maxima, in the bins with it: then the whole histogram).  The list begins again.
      if (R == 0 && tid == 0) ctl.n = 0u;
      cluster.sync();
      if (maxima) {
        masses = by_p;
        histogram(r, ctl, slice_count[0], slice_mass[0], masses, 0, Subset{0, 32, 0u});
        f = find_bin(ctl, slice_count[0], slice_mass[0], false, target, 0, Found{});
      }
    }
    kept = find_end(r, ctl, slice_count, slice_mass, !by_k, masses, target, f);
    if (by_k && by_p) {
      target = p_target(kept.mass);
      cluster.sync();  // find_end may come right from find_bin: every warp has read what it found before the next is told
      f = find_bin(ctl, slice_count[0], slice_mass[0], true, target, 0, Found{});
      kept = find_end(r, ctl, slice_count, slice_mass, true, true, target, f);
    }
  }

  // ---- kept weights by warp (runs of the row in order)
  const unsigned long long w_end = r.weight(value_of(kept.key));
  const uint32_t quota = w_end >= least ? kept.quota : 0u;
  unsigned long long mass = 0;
  uint32_t eq = 0;
  if (!by_k && !by_p && !least) {  // all of them
#pragma unroll 2
    for (int i = warp * chunk + lane; i < (warp + 1) * chunk; i += 32) {
      const uint4 v = seg[i];
#pragma unroll
      for (int m = 0; m < VE; ++m) mass += r.weight(element<BF16>(v, m));
    }
  } else {
    // A piece's weights are worked out side by side, whether kept or not, unless the whole
    // warp has none that is (what min-p drops lies below log2 of it, with some room).
    const float low = least ? fmaf(log2f(fminf(min_p, 1.0f)), 1.0001f, -0.001f) : -INFINITY;
    for (int i0 = warp * chunk; i0 < (warp + 1) * chunk; i0 += 32) {
      const int i = i0 + lane;
      uint4 v = make_uint4(kNone, kNone, kNone, kNone);
      if (i < (warp + 1) * chunk) v = seg[i];
      bool in[VE], any = false;
#pragma unroll
      for (int m = 0; m < VE; ++m) {
        const float x = element<BF16>(v, m);
        const uint32_t key = key_of(x);
        in[m] = key > kept.key && !((x - mx) * r.c_hi < low);
        any |= in[m];
        eq += key == kept.key && i < (warp + 1) * chunk;
      }
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int m = 0; m < VE; ++m) {
          const unsigned long long w = r.weight(element<BF16>(v, m));
          mass += in[m] && w >= least ? w : 0ull;
        }
      }
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
    const unsigned long long target = __umul64hi(u64, total);
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
          if (a.logp) a.logp[t] = log_share(x, w, total);
        }
        at += w;
      }
    }
    if (__any_sync(0xffffffffu, hit)) return;
    before += __shfl_sync(0xffffffffu, in, 31);
    eq_before += __shfl_sync(0xffffffffu, eq_in, 31);
  }
}

// CTAs of a row, a power of two.  Few rows are spread as wide as it goes, down to 16 KB a
// CTA; with more rows than the SMs take at once a CTA has up to 64 KB, as what it does for a
// cluster's sake is the same for less (in us, by 16 / 64 KB: one row of 5000 16.1 / 19.5; 256
// rows of 131072 in bf16 167 / 151, 500 of 20000 in fp32 178 / 85).
int cluster_of(int T, int V, bool bf16) {
  const int64_t bytes = static_cast<int64_t>(V) * (bf16 ? 2 : 4);
  int C = 1;
  while (C < kMaxCluster && (bytes > static_cast<int64_t>(C) * 65536 || (bytes > static_cast<int64_t>(C) * 16384 && static_cast<int64_t>(T) * C <= 152)))
    C *= 2;
  return C;
}

struct Plan {
  int C, chunk;
  size_t smem;
};
Plan plan_of(int T, int V, bool bf16) {
  const int VE = bf16 ? 8 : 4;
  Plan p;
  p.C = cluster_of(T, V, bf16);
  const int64_t vecs = (static_cast<int64_t>(V) + 2 * (VE - 1)) / VE + 1;  // wherever the row starts
  p.chunk = static_cast<int>((vecs + p.C * kWarps - 1) / (p.C * kWarps));
  p.smem = static_cast<size_t>(p.chunk) * kWarps * 16 + sizeof(Control) + static_cast<size_t>(kBins / p.C) * 2 * 12;
  return p;
}

}  // namespace

// what eight CTAs' shared memory holds
bool sample_supported(int V, bool bf16) { return V <= (bf16 ? 800000 : 400000) && plan_of(1, V, bf16).smem <= 227 * 1024; }

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  const Plan p = plan_of(a.T, a.V, a.bf16 != 0);
  void (*kernel)(SampleArgs, int) = a.bf16 ? k_sample<true> : k_sample<false>;
  static std::atomic<uint64_t> allowed[2];
  cudaError_t e = allow_smem(kernel, allowed[a.bf16 ? 1 : 0], 227 * 1024);
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
