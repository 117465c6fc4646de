// Attention of chunks of new tokens over the paged MX cache on the tensor
// cores: tcgen05 MMAs with the accumulators in tensor memory.
//
// What bounds it.  With heads of 128 a unit of 64 keys and 256 rows is 1024
// cycles of MMAs at their rate; it takes 1750: the 8-bit MMAs read Q again for
// every unit (64 KB of the 128 KB that a unit's operands are, at 128 bytes a
// cycle), which tensor memory, full, cannot hold, and the softmax's two warps a
// scheduler need about as long.  With heads of 64 the softmax alone bounds a
// unit (1560).  A segment costs 16 (10) units more: queries split into their
// two parts, the accumulator written out, the first keys of the next on their
// way through empty stages.  2048 new tokens behind 14336 take 414 us (1245
// TFLOP/s of 4 head_dim flops for each visible (row, key) pair, 64% of a plain
// bf16 product's), a prompt of 8192 510 us (1078).  Over an MXFP4 cache they take
// 574 and 689: V's warps turn K's codes into 8-bit ones as well.
//
// A tile is 256 rows (new tokens x the query heads of one KV head) as two MMA
// tiles of 128, A and B, that take turns: while the tensor cores work for one,
// the softmax of the other runs.  Roles (sixteen warps):
//   0-3, 4-7   softmax of A and of B, one row a thread; also its queries, the
//              rescaling of its accumulator and its output
//   8, 12      issuing the MMAs of A and of B
//   9          fetching codes and scales, by TMA and bulk copies
//   13         scales: K's into their place for the MMAs, V's for V's warps
//   10, 11, 14, 15  V: codes into the 16-bit operand, from and to shared memory
//              (and K's into 8-bit ones, where they are E2M1)
// (a scheduler runs the warps of one number modulo 4: each has two softmax warps and
// one or two of the others, whose loops have to fit its instruction cache together)
// For each unit of keys, S = Q K^T goes to tensor memory and from there to the
// softmax's registers, which frees it for the next unit's S; the softmax weights
// P go back to tensor memory, and O += P V reads them there.
//
// Arithmetic.  S is a block-scaled MMA on the cache's own codes and scales, so K
// is never widened.  A query row is split into two MXFP8 operands, q = hi + lo:
// hi is q on a grid of 4 significant bits, lo the rest (at most 5 bits) at a
// scale 2^-5 of hi's.  Together they hold bf16's 8 bits of every element down
// to 2^-13 of its block's largest, and 2^-21 of the largest below; two MMAs at
// the 8-bit rate cost what one bf16 MMA would.
// V varies its scale along N, which the block-scaled MMA cannot take, so V is
// widened: exactly, to f16 relative to the unit's largest V scale e, as long as
// the unit's scales lie within 2^15; P is then rounded to f16 (2^-11).  A unit
// with a wider spread takes bf16 for both (V exact, P 2^-8).  As in the few-rows
// kernel e joins the softmax's exponent: P = 2^(x + e - M) with M the running
// maximum of x + e, and the sum adds (sum of P) 2^-e.  M moves only when it
// would grow by more than 2^8, so O is seldom rescaled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <climits>
#include <cstdint>

#include "attn.cuh"
#include "kv.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int kRows = 256;
constexpr int kThreads = 512;
constexpr int kMaxCtas = 152;
constexpr int kMinUnits = 20;  // places of a CTA's stretch at least
// A segment's queries and output, in units (a prompt of 8192: 510 us with 16, 515 with
// 12, 520 with 20).  Heads of 64, whose segments cost 10, take the same: 8 prompts of up
// to 500: 35 us with 16, 41 with 10; a prompt of 8192: 445 and 431.
constexpr int kCost = 16;
// Least units of a split segment's part: a part costs queries and an output again
// (6 prompts of up to 662 with 10 KV heads: 55 us with 1, 32 with 4, 30 with 8 and 12;
// 256 new tokens over 4096, whose 32 segments are all there is to share out: 50, 50, 53,
// 57).
constexpr int kSnap = 8;
constexpr int kStages = 4;     // of K and of V
constexpr int kRawStages = 4;  // of codes on their way to V
constexpr int kMetaRing = 8;  // more units than can be between their scales' arrival and their softmax
// AttnCursor::settle, out of line, and the units of a whole stretch.
template <class Cursor>
__device__ __noinline__ bool settle(Cursor& c, const AttnArgs& a) {
  return c.settle(a);
}
template <class Cursor>
__device__ __forceinline__ int units_of(Cursor& c, const AttnArgs& a) {
  int n = 0;
  while (settle(c, a)) {
    const int k = c.take();
    n += k;
    c.pass(k);
  }
  return n;
}

// What the softmax and the MMA issuer need to know of a unit.
struct alignas(16) UnitMeta {
  int v_exp;  // exponent of its largest V scale
  int wide;   // V and P in bf16
  uint32_t bad;  // UnitKeys::bad
  float back;    // 2^-v_exp, or NaN where a V scale is
};
// A unit's keys to read, counted from its first, and its 16-key groups that are
// not there (a bit each).
struct UnitKeys {
  int lo, hi;
  uint32_t gone;
  uint32_t bad;  // of those, the ones that rows would see but for their page
};

template <int D>
struct Shape {
  // Keys of a unit.  Tensor memory has 512 columns: two S (one a key), two P
  // (half as many), two O (one an element) and the scales' 48.
  static constexpr int kUnit = 64;
  static constexpr uint32_t kQTile = 128 * D;                // one 8-bit operand
  static constexpr uint32_t kKStage = kUnit * D;
  static constexpr uint32_t kVPanel = kUnit * 128;           // 64 16-bit elements of each key
  static constexpr uint32_t kVStage = kVPanel * (D / 64);
  static constexpr uint32_t kQ = 0;                          // A hi, A lo, B hi, B lo
  static constexpr uint32_t kK = 4 * kQTile;
  static constexpr uint32_t kV = kK + kStages * kKStage;
  // as they come: V's codes (and K's where they are E2M1), K's scales, V's
  static constexpr uint32_t kRaw = kV + kStages * kVStage;
  static constexpr uint32_t kRawScales = kUnit * D, kScaleBytes = kUnit * (D / 32);
  static constexpr uint32_t kRawStage = (kRawScales + 2 * kScaleBytes + 1023) / 1024 * 1024;
  static constexpr uint32_t kBytes = kRaw + kRawStages * kRawStage;
  static_assert(kKStage % 1024 == 0 && kVPanel % 1024 == 0, "swizzle atoms");
  // tensor memory columns
  static constexpr uint32_t kS = 0, kP = 2 * kUnit;          // A, then B kUnit (kUnit / 2) on
  static constexpr uint32_t kScales = 3 * kUnit;             // of A and of B: Q hi, Q lo, K's stages, four each
  static constexpr uint32_t kScalesOf = 8 + 4 * kStages;
  static constexpr uint32_t kO = 512 - 2 * D;                // A, then B
  static_assert(kScales + 2 * kScalesOf <= kO, "tensor memory");
};
constexpr uint32_t kTmemColumns = 512;

struct Shared {
  uint64_t q_full[2], s_full[2], s_empty[2], p_full[2], p_empty[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], drain[2];
  uint64_t raw_full[kRawStages], raw_empty[kRawStages], meta_full[kRawStages];
  uint32_t tmem;
  volatile int failed;
  int last[2];
  UnitMeta meta[kMetaRing];
  uint32_t q_scale[2][128];  // a row's scale bytes
  alignas(16) uint4 rows[8][32][4];  // a warp's finished rows on their way to the output, 32 elements of each
  alignas(128) uint32_t k_scale[kStages][32][4];  // keys 32 j + lane, by lane
  UnitKeys keys[kRawStages];
  uint32_t units[kAttnScan];
};

// Functions that are not inlined here and below: the roles' unit loops have to
// fit the instruction caches together (timed with a loop of multiply-adds for each
// of an SM's four schedulers: full speed up to 512 of them, a quarter of it past
// 2048), so what a unit seldom needs lies outside of them.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  return attn_wait<false>(&sh.failed, bar, parity, a);
}

// The 128 threads of a tile's softmax meet.
__device__ __forceinline__ void tile_barrier(int x) { asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory"); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// E4M3 codes of two f16, to nearest even, saturating.
__device__ __forceinline__ uint32_t enc_e4m3x2_f16(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// 2^d twice, as f16 (subnormal below -14, 0 below -24; d <= 15) and as bf16
// times 2^112 (0 below the type's range).
__device__ __forceinline__ uint32_t f16_pow2x2(int d) {
  return (d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : 0x400u >> min(-14 - d, 31)) * 0x10001u;
}
__device__ __forceinline__ uint32_t bf16_pow2x2_112(int d) {
  return (d >= -238 ? static_cast<uint32_t>(127 + 112 + d) << 7 : 0u) * 0x10001u;
}
// An f16 pair that holds codes' values (no f16 subnormals but 0) as bf16 times
// 2^-112: the f16 exponent and mantissa moved to bf16's places.
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h) {
  return ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u);
}
// Four E2M1 codes (16 bits) as E4M3 codes: the magnitudes by a byte table.
__device__ __forceinline__ uint32_t e4m3_of_e2m1x4(uint32_t c) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, c & 0x7777u);
  const uint32_t twice = __byte_perm(c, 0u, 0x1100u);  // each byte next to itself
  return mag | ((twice << 4) & 0x00800080u) | (twice & 0x80008000u);
}

// Sixteen codes of one key, a lane's share.
template <bool E2M1>
struct Codes {
  static constexpr int kWords = E2M1 ? 2 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (E2M1) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  // elements 2i, 2i + 1
  __device__ __forceinline__ uint32_t pair(int i) const {
    if constexpr (E2M1) return f16x2_of_e2m1x2((w[i / 4] >> (8 * (i % 4))) & 0xFFu);
    else return f16x2_of_e4m3x2((w[i / 2] >> (16 * (i % 2))) & 0xFFFFu);
  }
};

// n columns (a multiple of 8) of a lane from tensor memory, not yet waited for.
template <int kN>
__device__ __forceinline__ void tmem_load(uint32_t col, uint32_t (&v)[kN]) {
  static_assert(kN % 16 == 0, "");
#pragma unroll
  for (int c = 0; c + 32 <= kN; c += 32) tmem_ld_32x32b_x32(col + c, reinterpret_cast<uint32_t(&)[32]>(v[c]));
  if constexpr (kN % 32 != 0) tmem_ld_32x32b_x16(col + kN / 32 * 32, reinterpret_cast<uint32_t(&)[16]>(v[kN / 32 * 32]));
}

// A lane's keys of a unit to the V operand (its pieces of key r0 + r at to0 and
// to1, 128 bytes a key), those outside the unit's keys to read as zeros; kWide in
// bf16.  The unit loop has the common case, f16 and all keys, itself.
template <int kUnit, int kStep, int D, bool E2M1, bool kWide>
__device__ __noinline__ void widen(const uint8_t* codes, const uint8_t* scales, uint8_t* to0, uint8_t* to1, UnitMeta meta,
                                   UnitKeys keys, int r0) {
  constexpr int kRowBytes = E2M1 ? D / 2 : D;
#pragma unroll 1
  for (int r = 0; r < kUnit; r += kStep) {
    Codes<E2M1> v;
    v.load(codes + r * kRowBytes);
    const int k = r + r0;
    if (k < keys.lo || k >= keys.hi || (keys.gone >> (k / 16) & 1u)) v.clear();
    const int d = min(scales[r * (D / 32)] - 127 - meta.v_exp, 15);
    const uint32_t f = kWide ? bf16_pow2x2_112(d) : f16_pow2x2(d);
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = kWide ? mul_bf16x2(bf16x2_of_f16x2(v.pair(e)), f) : mul_f16x2(v.pair(e), f);
    *reinterpret_cast<uint4*>(to0 + r * 128) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(to1 + r * 128) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Sixteen finished elements of row oh of the output, and its lse.
template <int D>
__device__ __forceinline__ void put(const AttnArgs& a, int64_t oh, int c, const float (&v)[16], float inv) {
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + oh * D + c);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    dst[i] = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                        pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
}
__device__ __forceinline__ void put_lse(const AttnArgs& a, int64_t oh, float M, float L) {
  if (a.lse) a.lse[oh] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}
// Four elements of a row of a part: the same elements of all rows side by side.
template <int D>
__device__ __forceinline__ float4* part_at(const AttnArgs& a, int slot, int d4, int row) {
  return reinterpret_cast<float4*>(a.part_o) + (static_cast<int64_t>(slot) * (D / 4) + d4) * kRows + row;
}

// A tile's queries as two MXFP8 operands and their scales, by the 128 threads of
// its softmax: eight elements a lane at a time, four lanes a block.
template <int D>
__device__ __noinline__ void load_queries(const AttnArgs& a, Shared& sh, uint8_t* base, int x, int q0, int head, int row0,
                                          int rows) {
  using Sh = Shape<D>;
  constexpr uint32_t tmem = 0;
  const int lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(threadIdx.x & 96) << 16;
  constexpr int kPieces = D / 8;     // sixteen bytes of bf16
  constexpr int kStep = 128 / kPieces;  // rows of the 128 threads
  // Pieces converted side by side, and on their way behind them (a prompt of 8192:
  // 510 us; 1 and 4: 516; 4 and 4: 513; with 2 and 8 the unit loop's registers spill:
  // 554).
  constexpr int kTogether = 2, kAhead = 4;
  const int p = threadIdx.x % kPieces, r0 = (threadIdx.x & 127) / kPieces;
  uint8_t* hi_base = base + Sh::kQ + 2 * x * Sh::kQTile;
  auto load = [&](int r) {
    const int R = row0 + r;
    if (r >= 128 || R >= rows) return make_uint4(0u, 0u, 0u, 0u);
    const int tok = a.group_div.of(R);
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                static_cast<int64_t>(q0 + tok) * a.q_stride +
                                                static_cast<int64_t>(head * a.group + (R - tok * a.group)) * D) + p);
  };
  uint4 queue[kAhead + kTogether];
#pragma unroll
  for (int n = 0; n < kAhead; ++n) queue[n] = load(r0 + n * kStep);
#pragma unroll 1
  for (int rr = r0; rr < 128; rr += kTogether * kStep) {
#pragma unroll
    for (int n = 0; n < kTogether; ++n) queue[kAhead + n] = load(rr + (kAhead + n) * kStep);
#pragma unroll
    for (int n = 0; n < kTogether; ++n) {
      const int r = rr + n * kStep;
      const uint32_t w[4] = {queue[n].x, queue[n].y, queue[n].z, queue[n].w};
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = __vmaxu2(amax, w[k] & 0x7FFF7FFFu);
      amax = max(amax & 0xFFFFu, amax >> 16);
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the block's largest element lands in [2^7, 2^8): hi's rounding error
      // is then at most 2^3 and 2^5 times it stays below E4M3's 448
      const int s = max(static_cast<int>(amax >> 7) - 127 - 7, -122);
      // a block with an infinity or NaN has no scores
      const float down = amax >= 0x7F80u ? __uint_as_float(0x7FC00000u) : pow2_neg(s);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          // in f16 (exact down to 2^-25 of the block's largest, which lo does not hold)
          const uint32_t x = pack_f16(__uint_as_float(w[k + m] << 16) * down, __uint_as_float(w[k + m] & 0xFFFF0000u) * down);
          h[m] = enc_e4m3x2_f16(x);
          l[m] = enc_e4m3x2_f16(mul_f16x2(sub_f16x2(x, f16x2_of_e4m3x2(h[m])), 0x50005000u));  // 32
        }
        hi[k / 2] = __byte_perm(h[0], h[1], 0x5410);
        lo[k / 2] = __byte_perm(l[0], l[1], 0x5410);
      }
      const uint32_t at = D == 128 ? r * 128 + (((p >> 1) ^ (r & 7)) << 4) + (p & 1) * 8
                                   : r * 64 + (((p >> 1) ^ ((r >> 1) & 3)) << 4) + (p & 1) * 8;
      *reinterpret_cast<uint2*>(hi_base + at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(hi_base + Sh::kQTile + at) = make_uint2(lo[0], lo[1]);
      if ((p & 3) == 0) reinterpret_cast<uint8_t*>(&sh.q_scale[x][r])[p >> 2] = static_cast<uint8_t>(s + 127);
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) queue[n] = queue[n + kTogether];
  }
  fence_proxy_async_shared();
  tile_barrier(x);
  // scales: row 32 j + lane in column j, the same in every lane quarter
  const uint32_t col = tmem + lanes + Sh::kScales + Sh::kScalesOf * x;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = sh.q_scale[x][32 * j + lane];
  tmem_st_32x32b_x4(col, w[0], w[1], w[2], w[3]);
  constexpr uint32_t kFive = D == 128 ? 0x05050505u : 0x0505u;
  tmem_st_32x32b_x4(col + 4, w[0] - kFive, w[1] - kFive, w[2] - kFive, w[3] - kFive);
  tmem_st_wait();
  tc_fence_before();
  warp_arrive(&sh.q_full[x]);
}

// S columns outside [lo, hi), and those of the 16-column groups in `bad`, to
// -inf, in a unit at the edge of what rows see.
template <int kColumns>
__device__ __noinline__ void mask_scores(uint32_t s_col, int lo, int hi, uint32_t bad) {
#pragma unroll 1
  for (int c = 0; c < kColumns; c += 16) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(s_col + c, v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i >= hi || c + i < lo || (bad >> (c / 16) & 1u)) v[i] = 0xFF800000u;
    tmem_st_32x32b_x16(s_col + c, v);
  }
  tmem_st_wait();
}
// O times f, when the running maximum has moved.
template <int D>
__device__ __noinline__ void rescale(uint32_t o_col, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld_32x32b_x16(o_col + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tmem_st_32x32b_x16(o_col + c, o);
  }
}

// A row of a split segment from its parts, in key order.
template <int D>
__device__ __forceinline__ void join_parts(const AttnArgs& a, AttnParts p, int row, int64_t oh) {
  auto ml_of = [&](int i) { return __ldcg(&a.part_ml[attn_slot(p.first + i, i == 0) * kRows + row]); };
  float M = -INFINITY;
  for (int i = 0; i < p.parts; ++i) M = fmaxf(M, ml_of(i).x);
  const float from = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  for (int i = 0; i < p.parts; ++i) {
    const float2 ml = ml_of(i);
    L = fmaf(ml.y, exp2_approx(ml.x - from), L);
  }
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.0f;
#pragma unroll 2
    for (int i = 0; i < p.parts; ++i) {
      const float w = exp2_approx(ml_of(i).x - from);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = __ldcg(part_at<D>(a, attn_slot(p.first + i, i == 0), c / 4 + k, row));
        f[4 * k] = fmaf(v.x, w, f[4 * k]), f[4 * k + 1] = fmaf(v.y, w, f[4 * k + 1]);
        f[4 * k + 2] = fmaf(v.z, w, f[4 * k + 2]), f[4 * k + 3] = fmaf(v.w, w, f[4 * k + 3]);
      }
    }
    put<D>(a, oh, c, f, L == 0.0f ? 0.0f : 1.0f / L);
  }
  put_lse(a, oh, M, L);
}

// A tile's rows when its stretch of the segment ends: to the output, or (slot >=
// 0) as a part, and then the last part to arrive joins them all.
template <int D>
__device__ __noinline__ void write_rows(const AttnArgs& a, Shared& sh, uint32_t o_col, int x, int slot, AttnParts parts,
                                        int64_t oh, bool ok, bool warp_valid, bool valid, float m, float l) {
  const int row = threadIdx.x & 127;
  const int lane = threadIdx.x & 31;
  if (ok && warp_valid && slot < 0) {
    // 32 elements of every row at a time by way of shared memory: a warp's store
    // is then eight rows of 64 bytes, not 32 of 16 (64 new tokens over 256 keys
    // of 114 sequences and 8 KV heads: 128 -> 115 us)
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint4(&stage)[32][4] = sh.rows[threadIdx.x >> 5];
    // of the rows that the lane stores
    int64_t at[4];
    bool there[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at[i] = __shfl_sync(0xffffffffu, oh, 8 * i + lane / 4) * D + lane % 4 * 8;
      there[i] = __shfl_sync(0xffffffffu, static_cast<int>(valid), 8 * i + lane / 4);
    }
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(o_col + c, v);
      tmem_ld_wait();
      // a row without a visible key never had its accumulator's weights defined
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = l == 0.0f ? 0u : pack_bf16(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        stage[lane][i ^ (lane >> 1 & 3)] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + lane / 4;
        if (there[i]) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at[i] + c) = stage[r][lane % 4 ^ (r >> 1 & 3)];
      }
      __syncwarp();
    }
    if (valid) put_lse(a, oh, m, l);
  } else if (ok && warp_valid) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(o_col + c, v);
      tmem_ld_wait();
      float f[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = l == 0.0f ? 0.0f : __uint_as_float(v[i]);
      if (valid) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *part_at<D>(a, slot, c / 4 + i, 128 * x + row) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
      __syncwarp();
    }
    if (valid) a.part_ml[slot * kRows + 128 * x + row] = make_float2(m, l);
  }
  if (slot < 0) return;
  // also after a wait that ran out: the counters are zero for the next call
  tile_barrier(x);
  unsigned* counter = &a.arrived[2 * parts.first + x];
  if (row == 0) {
    sh.last[x] = attn_arrive(counter) == static_cast<unsigned>(parts.parts - 1);
    if (sh.last[x]) *counter = 0u;
  }
  tile_barrier(x);
  if (sh.last[x] && ok && valid) {
    join_parts<D>(a, parts, 128 * x + row, oh);
  }
  __syncwarp();
}

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads, 1) k_attn_chunk(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                                                              const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<D>;
  constexpr int kUnit = Sh::kUnit;
  using Cursor = AttnCursor<kRows, kUnit, kCost, kSnap>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same for the warp, and known to be
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 4);  // one arrival a warp, here and below
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_empty[i]), 4);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.p_empty[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), E2M1 ? 5 : 2);  // scales, and codes by TMA or by V's warps
      mbar_init(smem_u32(&sh.k_empty[i]), 2);  // by A's MMAs and B's
      mbar_init(smem_u32(&sh.v_full[i]), 4);
      mbar_init(smem_u32(&sh.v_empty[i]), 2);
    }
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(smem_u32(&sh.raw_full[i]), 1);
      mbar_init(smem_u32(&sh.raw_empty[i]), 5);  // V's warps, and the scales'
      mbar_init(smem_u32(&sh.meta_full[i]), 1);
    }
    mbar_init(smem_u32(&sh.drain[0]), 1);
    mbar_init(smem_u32(&sh.drain[1]), 1);
    sh.failed = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&sh.tmem), kTmemColumns);
    tmem_relinquish();
  }
  const AttnShare share = attn_share<kRows, kUnit, kCost, kThreads, true>(a, sh.units);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all of tensor memory is this CTA's
  Cursor cur;
  cur.template start<true>(a, share);
  if (warp < 8) {
    // ================================================================ softmax
    const int x = warp >> 2;                       // tile A or B
    const int row = tid & 127;                     // the thread's row of it
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + Sh::kS + kUnit * x, p_col = tmem + lanes + Sh::kP + kUnit / 2 * x;
    const uint32_t o_col = tmem + lanes + Sh::kO + D * static_cast<uint32_t>(x);
    uint32_t unit = 0, s_phase = 0, p_phase = 0;
    bool ok = true;

    sh.q_scale[x][row] = 0u;
    tile_barrier(x);
    auto queries_of = [&](const Cursor& c) {
      const int rows = c.s.n * a.group, row0 = c.tile * kRows + 128 * x;
      if (row0 < rows) load_queries<D>(a, sh, base, x, c.s.q0, c.head, row0, rows);
    };
    bool more = settle(cur, a);
    if (more) queries_of(cur);
    while (more) {
      const int take = cur.take();
      const int rows = cur.s.n * a.group;
      const int row0 = cur.tile * kRows + 128 * x;
      Cursor ahead;
      auto to_next = [&]() {  // and its queries
        ahead = cur;
        ahead.pass(take);
        more = settle(ahead, a);
        if (more) queries_of(ahead);
      };
      if (row0 < rows) {
        const int R = row0 + row;
        const bool valid = R < rows;
        const int tok = valid ? a.group_div.of(R) : 0;
        const int at = cur.s.kv - cur.s.n + tok;
        // rows past the last see everything: their queries are zero
        const int hi = !valid ? INT_MAX : a.causal ? min(cur.s.kv, max(at + 1, 0)) : cur.s.kv;
        const int lo = valid && a.window > 0 ? attn_row_lo(a, at) : 0;
        const int all_hi = __reduce_min_sync(0xffffffffu, hi), all_lo = __reduce_max_sync(0xffffffffu, lo);
        const bool warp_valid = row0 + 32 * (warp & 3) < rows;
        const float scale = a.scale_log2;
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (int j = 0; j < take; ++j) {
          if (ok && !wait(sh, &sh.s_full[x], s_phase, a)) ok = false;
          s_phase ^= 1u;
          tc_fence_after();
          const UnitMeta meta = sh.meta[(unit + j) % kMetaRing];
          const int key0 = cur.t.first + (cur.place + j) * kUnit;
          uint32_t v[kUnit];
          __syncwarp();
          // Lanes may differ in whether their wait ran out, and what follows is for
          // the whole warp (tensor memory, votes): so what leads there is either the
          // same for all lanes or voted on (the vote: 412 -> 414 us in the header's
          // chunk), and a warp goes on with whatever it finds; its rows are not
          // written at the end.
          if (warp_valid) {
            if (__any_sync(0xffffffffu, key0 + kUnit > all_hi || key0 < all_lo || meta.bad != 0))
              mask_scores<kUnit>(s_col, lo - key0, hi - key0, meta.bad);
            tmem_load<kUnit>(s_col, v);
            tmem_ld_wait();
          }
          tc_fence_before();
          warp_arrive(&sh.s_empty[x]);
          // for the last unit's P to have been read, and O written; asked for
          // ahead of the exponentials, which hide the answer's way
          bool read = j == 0;
          auto wait_values = [&]() {
            if (!read && ok) ok = wait(sh, &sh.p_empty[x], p_phase, a);
            read = true;
            __syncwarp();
            tc_fence_after();
          };
          if (warp_valid) {
            float t4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t4[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[4 + k]));
#pragma unroll
            for (int i = 8; i < kUnit; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) t4[k] = max3(t4[k], __uint_as_float(v[i + k]), __uint_as_float(v[i + 4 + k]));
            }
            const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            const float e = static_cast<float>(meta.v_exp);
            const float joint = fmaf(top, scale, e);
            if (__any_sync(0xffffffffu, joint > m + 8.0f)) {
              const float to = fmaxf(m, joint);
              const float f = to == -INFINITY ? 1.0f : exp2_approx(m - to);
              // O holds something but zeros once a row has seen a key
              const bool seen = __any_sync(0xffffffffu, m != -INFINITY);
              m = to;
              l *= f;
              if (seen) {
                wait_values();
                rescale<D>(o_col, f);
              }
            }
            if (!read) read = mbar_try_wait(smem_u32(&sh.p_empty[x]), p_phase);
            const float off = m == -INFINITY ? 0.0f : e - m;
            const float2 scale2 = make_float2(scale, scale), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            auto weights = [&](auto pack) {
#pragma unroll
              for (int i = 0; i < kUnit; i += 2) {
                const float2 z = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), scale2, off2);
                const float2 w = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], w);
                v[i / 2] = pack(w);
              }
            };
            if (__builtin_expect(meta.wide, 0)) weights([](float2 w) { return pack_bf16(w.x, w.y); });
            else weights([](float2 w) { return pack_f16(w.x, w.y); });
            const float2 all = add2(sum[0], sum[1]);
            l = fmaf(all.x + all.y, meta.back, l);
            wait_values();
            tmem_st_32x32b_x32(p_col, reinterpret_cast<uint32_t(&)[32]>(v[0]));
            tmem_st_wait();
          } else {
            wait_values();
          }
          if (j > 0) p_phase ^= 1u;
          tc_fence_before();
          warp_arrive(&sh.p_full[x]);
        }
        // the last scores are done: the next segment's queries may come
        to_next();

        if (ok) ok = wait(sh, &sh.p_empty[x], p_phase, a);
        p_phase ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const int64_t oh = static_cast<int64_t>(cur.s.q0 + tok) * (a.n_kv_heads * a.group) + cur.head * a.group + (R - tok * a.group);
        const bool whole = take == cur.t.units;
        AttnParts parts{};
        if (!whole) parts = attn_parts<kSnap>(share, cur.u - cur.place, cur.t.units);
        write_rows<D>(a, sh, o_col, x, whole ? -1 : attn_slot(blockIdx.x, cur.place == 0), parts, oh, ok, warp_valid, valid, m, l);
      } else {
        to_next();  // this segment has no tile B
      }
      unit += take;
      cur = ahead;
    }
  } else if (warp & 2) {
    // ================================================================ V, and K's scales
    constexpr int kShares = D / 16;            // lanes of a key: sixteen elements each
    constexpr int kKeysPerIt = 128 / kShares;  // over the four warps
    constexpr int kRowBytes = E2M1 ? D / 2 : D;
    constexpr int kPieceBytes = kRowBytes / kShares;
    constexpr int kBlocks = D / 32;
    const int dw = (warp & 1) + (warp >= 12 ? 2 : 0);
    // Lanes 0-15 take the first 64 elements of their keys and, with 128, lanes
    // 16-31 the second: eight lanes of a store then lie in two rows of one
    // panel, which touches all banks.
    const int part = lane % 4 + (D == 128 ? lane / 16 * 4 : 0);
    const int r0 = dw * (32 / kShares) + (D == 128 ? lane % 16 / 4 : lane / 4);
    // a lane's two 16-byte pieces of a V row; kKeysPerIt is a multiple of 8, so
    // the swizzle is the same for all its keys
    const uint32_t v_at = (part / 4) * Sh::kVPanel + r0 * 128;
    const uint32_t v_at0 = v_at + (((part % 4 * 2) ^ (r0 & 7)) << 4), v_at1 = v_at + (((part % 4 * 2 + 1) ^ (r0 & 7)) << 4);
    const uint32_t k_at = D == 128 ? r0 * 128 + ((part ^ (r0 & 7)) << 4) : r0 * 64 + ((part ^ ((r0 >> 1) & 3)) << 4);
    const int n = units_of(cur, a);
    Ring<kStages> ring;
    Ring<kRawStages> raw;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      bool ok = wait(sh, &sh.raw_full[raw.stage], raw.phase, a) && wait(sh, &sh.meta_full[raw.stage], raw.phase, a);
      if (E2M1 && ok) ok = wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
      if (ok) ok = wait(sh, &sh.v_empty[ring.stage], ring.phase ^ 1u, a);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const UnitMeta meta = sh.meta[static_cast<uint32_t>(i) % kMetaRing];
      const uint8_t* codes = base + Sh::kRaw + raw.stage * Sh::kRawStage + r0 * kRowBytes + part * kPieceBytes;
      const uint8_t* scales = base + Sh::kRaw + raw.stage * Sh::kRawStage + Sh::kRawScales + Sh::kScaleBytes + r0 * kBlocks + part / 2;
      uint8_t* v_to = base + Sh::kV + ring.stage * Sh::kVStage;
      const UnitKeys keys = sh.keys[raw.stage];
      const bool cut = keys.lo > 0 || keys.hi < kUnit || keys.gone != 0;
      if (E2M1) {
        const uint8_t* k_codes = codes + kUnit * kRowBytes;
        uint8_t* k_to = base + Sh::kK + ring.stage * Sh::kKStage + k_at;
#pragma unroll 1
        for (int r = 0; r < kUnit; r += kKeysPerIt) {
          const uint2 c = *reinterpret_cast<const uint2*>(k_codes + r * kRowBytes);
          *reinterpret_cast<uint4*>(k_to + r * D) =
              make_uint4(e4m3_of_e2m1x4(c.x), e4m3_of_e2m1x4(c.x >> 16), e4m3_of_e2m1x4(c.y), e4m3_of_e2m1x4(c.y >> 16));
        }
        fence_proxy_async_shared();
        warp_arrive(&sh.k_full[ring.stage]);
      }
      if (__builtin_expect(meta.wide, 0)) {
        widen<kUnit, kKeysPerIt, D, E2M1, true>(codes, scales, v_to + v_at0, v_to + v_at1, meta, keys, r0);
      } else if (__builtin_expect(cut, 0)) {
        widen<kUnit, kKeysPerIt, D, E2M1, false>(codes, scales, v_to + v_at0, v_to + v_at1, meta, keys, r0);
      } else {
#pragma unroll 2
        for (int r = 0; r < kUnit; r += kKeysPerIt) {
          Codes<E2M1> v;
          v.load(codes + r * kRowBytes);
          const uint32_t f = f16_pow2x2(scales[r * kBlocks] - 127 - meta.v_exp);
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = mul_f16x2(v.pair(e), f);
          *reinterpret_cast<uint4*>(v_to + v_at0 + r * 128) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(v_to + v_at1 + r * 128) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      fence_proxy_async_shared();
      warp_arrive(&sh.v_full[ring.stage]);
      warp_arrive(&sh.raw_empty[raw.stage]);
      ring.next();
      raw.next();
    }
  } else {
    if (warp == 8 || warp == 12) {
      if (elect_one()) {
      // ================================================================ MMAs
      const uint32_t x = warp == 8 ? 0 : 1;
      // V is MN-major: 64-element panels along N lie kVPanel apart (leading
      // offset), eight-key groups 1024 bytes (stride)
      const uint32_t q_lo = desc_lo_sw128(smem_u32(base + Sh::kQ) + 2 * x * Sh::kQTile), k_lo = desc_lo_sw128(smem_u32(base + Sh::kK));
      const uint32_t v_lo = ((smem_u32(base + Sh::kV) >> 4) & 0x3FFFu) | ((Sh::kVPanel >> 4) << 16);
      constexpr uint32_t kQkHi = D == 128 ? kDescHiSw128 : kDescHiSw64;
      const uint32_t s_col = tmem + Sh::kS + kUnit * x, p_col = tmem + Sh::kP + kUnit / 2 * x, o_col = tmem + Sh::kO + D * x;
      const uint32_t q_sf = tmem + Sh::kScales + Sh::kScalesOf * x;
      uint32_t q_phase = 0, p_phase = 0, s_phase = 1;  // S is empty at first
      uint32_t unit = 0;
      bool ok = true;
      Ring<kStages> kr, vr;  // the next stage to take
      while (ok && settle(cur, a)) {
        const int take = cur.take();
        const bool active = cur.s.n * a.group - cur.tile * kRows > 128 * static_cast<int>(x);
        if (active) {
          ok = wait(sh, &sh.q_full[x], q_phase, a);
          q_phase ^= 1u;
        }
        // step j: S of unit j + 1 as soon as the last one is in the softmax's
        // registers, then O += P V of unit j
#pragma unroll 1
        for (int j = -1; j < take && ok; ++j) {
          if (j + 1 < take) {
            ok = wait(sh, &sh.k_full[kr.stage], kr.phase, a);
            if (!ok) break;
            if (active) {
              const uint32_t k_sf = q_sf + 8u + 4u * kr.stage;
              tmem_copy_scales(k_sf, smem_u32(&sh.k_scale[kr.stage][0][0]));
              ok = wait(sh, &sh.s_empty[x], s_phase, a);
              if (!ok) break;
              s_phase ^= 1u;
              tc_fence_after();
              const uint32_t k = k_lo + ((kr.stage * Sh::kKStage) >> 4);
#pragma unroll 1
              for (uint32_t part = 0; part < 2; ++part) {
#pragma unroll
                for (uint32_t b = 0; b < D / 32; ++b)
                  mma_mxf8f6f4_lo(s_col, q_lo + ((part * Sh::kQTile) >> 4) + 2u * b, k + 2u * b, kQkHi,
                                  idesc_mx(kFmtE4M3, kFmtE4M3, 128, kUnit, b, b), q_sf + 4u * part, k_sf, (part | b) != 0);
              }
              mma_commit(smem_u32(&sh.s_full[x]));
              mma_commit(smem_u32(&sh.k_empty[kr.stage]));
            } else {
              mbar_arrive(smem_u32(&sh.k_empty[kr.stage]));
            }
            kr.next();
          }
          if (j >= 0) {
            ok = wait(sh, &sh.v_full[vr.stage], vr.phase, a);
            if (ok && active) ok = wait(sh, &sh.p_full[x], p_phase, a);
            if (!ok) break;
            if (active) {
              p_phase ^= 1u;
              tc_fence_after();
              const uint32_t idesc = idesc_f16(sh.meta[unit % kMetaRing].wide != 0, true, 128, D);
              const uint32_t v = v_lo + ((vr.stage * Sh::kVStage) >> 4);
#pragma unroll
              for (uint32_t k = 0; k < kUnit / 16; ++k)
                mma_f16_ts(o_col, p_col + 8u * k, v + ((k * 2048u) >> 4), kDescHiSw128, idesc, (j | static_cast<int>(k)) != 0);
              mma_commit(smem_u32(&sh.p_empty[x]));
              mma_commit(smem_u32(&sh.v_empty[vr.stage]));
            } else {
              mbar_arrive(smem_u32(&sh.v_empty[vr.stage]));
            }
            vr.next();
            ++unit;
          }
        }
        cur.pass(take);
      }
      // every MMA issued has completed before tensor memory is released
      mma_commit(smem_u32(&sh.drain[x]));
      mbar_wait(smem_u32(&sh.drain[x]), 0, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ================================================================ fetching
      // K's codes, V's, K's scales and V's, in boxes of a.box_keys keys (16, 32
      // or 64: what divides a page; a copy costs the same whatever its size: with
      // pages of 64 and the arithmetic taken out, 2048 tokens behind 14336 took
      // 313 us in boxes of 64 and 414 in boxes of 16), a lane a box.  A box that
      // is not there is read past the codes' end, which fills zeros, and its
      // scales are not read.
      constexpr int kGroups = kUnit / 16, kBlocks = D / 32;
      constexpr uint32_t kCodeBytes = kUnit * (E2M1 ? D / 2 : D);  // of K or V
      const int group = lane % kGroups, kind = lane / kGroups;  // of 16 keys
      const bool leads = 16 * group % a.box_keys == 0;          // a box
      AttnWalk<kUnit> walk;
      const int none = a.num_pages * a.n_kv_heads * a.page_size;
      if (lane < 2) prefetch_tensormap(lane == 0 ? &k_map : &v_map);
      Ring<kStages> ring;
      Ring<kRawStages> raw;
      int issued = 0;
      bool ok = true;
      while (ok && settle(cur, a)) {
        const int take = cur.take();
        walk.start(a, cur, group);
#pragma unroll 1
        for (int j = 0; j < take; ++j) {
          uint32_t here, bad;
          const int row = walk.box(a, cur.head, group, here, bad);
          const uint32_t boxes = __ballot_sync(0xffffffffu, leads && row >= 0) & ((1u << kGroups) - 1);
          if (!E2M1) ok = wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
          if (ok) ok = wait(sh, &sh.raw_empty[raw.stage], raw.phase ^ 1u, a);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t raw_bar = smem_u32(&sh.raw_full[raw.stage]);
          const uint32_t k_bar = E2M1 ? raw_bar : smem_u32(&sh.k_full[ring.stage]);
          if (lane == 0) {
            sh.keys[raw.stage] = UnitKeys{walk.lo, walk.hi, here ^ ((1u << kGroups) - 1), bad};
            mbar_arrive_expect_tx(raw_bar, (E2M1 ? 2 : 1) * kCodeBytes + 2 * __popc(boxes) * (a.box_keys * kBlocks));
            if (!E2M1) mbar_arrive_expect_tx(k_bar, kCodeBytes);
          }
          __syncwarp();
          const uint32_t to = smem_u32(base + Sh::kRaw + raw.stage * Sh::kRawStage);
          if (leads && kind < 2) {
            const uint32_t k_to = E2M1 ? to + kCodeBytes : smem_u32(base + Sh::kK + ring.stage * Sh::kKStage);
            tma_load_2d((kind == 0 ? k_to : to) + group * (kCodeBytes / kGroups), kind == 0 ? &k_map : &v_map, 0, row < 0 ? none : row,
                        kind == 0 ? k_bar : raw_bar);
          } else if (leads && kind < 4 && row >= 0) {
            bulk_load(to + Sh::kRawScales + (kind - 2) * Sh::kScaleBytes + group * 16 * kBlocks,
                      (kind == 2 ? a.k_scales : a.v_scales) + static_cast<int64_t>(row) * kBlocks, a.box_keys * kBlocks, raw_bar);
          }
          __syncwarp();
          ++issued;
          ring.next();
          raw.next();
          walk.step(a);
        }
        cur.pass(take);
      }
      // the last fills have landed before the CTA exits, also where a wait of
      // the others ran out
      for (int i = issued > kRawStages ? issued - kRawStages : 0; i < issued; ++i)
        mbar_wait(smem_u32(&sh.raw_full[i % kRawStages]), (i / kRawStages) & 1u, 100000000ull);
      for (int i = issued > kStages ? issued - kStages : 0; i < issued && !E2M1; ++i)
        mbar_wait(smem_u32(&sh.k_full[i % kStages]), (i / kStages) & 1u, 100000000ull);
      __syncwarp();
    } else if (warp == 13) {
      // ================================================================ scales
      constexpr int kWords = kUnit / 32, kBlocks = D / 32;
      const int n = units_of(cur, a);
      Ring<kStages> ring;
      Ring<kRawStages> raw;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        bool ok = wait(sh, &sh.raw_full[raw.stage], raw.phase, a) && wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const UnitKeys keys = sh.keys[raw.stage];
        const uint8_t* from = base + Sh::kRaw + raw.stage * Sh::kRawStage + Sh::kRawScales;
        // keys 32 j + lane: a row's scale bytes
        uint32_t ks[kWords], top = 0, low = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const int r = 32 * j + lane;
          uint32_t w;
          if constexpr (kBlocks == 4) {
            ks[j] = reinterpret_cast<const uint32_t*>(from)[r];
            w = reinterpret_cast<const uint32_t*>(from + Sh::kScaleBytes)[r];
          } else {
            ks[j] = reinterpret_cast<const uint16_t*>(from)[r];
            w = reinterpret_cast<const uint16_t*>(from + Sh::kScaleBytes)[r];
          }
          if (r < keys.lo || r >= keys.hi || (keys.gone >> (r / 16) & 1u)) w = 0u;
          top = __vmaxu4(top, w);
          low = __vminu4(low, w | __vcmpeq4(w, 0u));
        }
        *reinterpret_cast<uint2*>(&sh.k_scale[ring.stage][lane][0]) = make_uint2(ks[0], ks[1]);
        static_assert(kWords == 2, "");
        fence_proxy_async_shared();
        // V's largest scale, and the smallest of a block that is not zero
        top = max(max(top & 0xFFu, (top >> 8) & 0xFFu), max((top >> 16) & 0xFFu, top >> 24));
        low = min(min(low & 0xFFu, (low >> 8) & 0xFFu), min((low >> 16) & 0xFFu, low >> 24));
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) {
          UnitMeta meta;
          meta.v_exp = min(max(static_cast<int>(top) - 127, -100), 126);
          meta.bad = keys.bad;
          meta.back = __uint_as_float(top == 255u ? 0x7FC00000u : static_cast<uint32_t>(127 - meta.v_exp) << 23);
          meta.wide = meta.v_exp - (static_cast<int>(low) - 127) > 15;
          sh.meta[static_cast<uint32_t>(i) % kMetaRing] = meta;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.k_full[ring.stage]));
          mbar_arrive(smem_u32(&sh.meta_full[raw.stage]));
          mbar_arrive(smem_u32(&sh.raw_empty[raw.stage]));
        }
        ring.next();
        raw.next();
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(sh.tmem, kTmemColumns);
}

template <int D, bool E2M1>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  constexpr int kSmem = Shape<D>::kBytes + 1024;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int sms = 0, dev = 0;
  cudaError_t e = attn_sm_count(&sms);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_attn_chunk<D, E2M1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  // K's E4M3 rows are an MMA operand as they are, swizzled on their way; the
  // codes that pass through V's warps keep their order
  CUtensorMap k_map, v_map;
  constexpr int kRowBytes = E2M1 ? D / 2 : D;
  e = attn_code_map(&k_map, a, a.k_codes, kRowBytes, !E2M1);
  if (e == cudaSuccess) e = attn_code_map(&v_map, a, a.v_codes, kRowBytes, false);
  if (e != cudaSuccess) return e;
  k_attn_chunk<D, E2M1><<<sms < kMaxCtas ? sms : kMaxCtas, kThreads, kSmem, s>>>(a, k_map, v_map);
  return cudaGetLastError();
}

}  // namespace

size_t attn_chunk_part_bytes(int head_dim) {
  return static_cast<size_t>(2) * kMaxCtas * kRows * (sizeof(float2) + sizeof(float) * head_dim);
}

cudaError_t launch_attn_chunk(AttnArgs a, cudaStream_t s) {
  a.min_units = kMinUnits;
  a.part_o = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2) * kMaxCtas * kRows);
  if (a.head_dim == 128) return a.e2m1 ? launch<128, true>(a, s) : launch<128, false>(a, s);
  return a.e2m1 ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace mxk
