// Attention of chunks of new tokens over the paged MX cache on the tensor
// cores: tcgen05 MMAs with the accumulators in tensor memory, bound by the
// MMAs (4 * head_dim flops for each visible (row, key) pair).
//
// A tile is 256 rows (new tokens x the query heads of one KV head) as two MMA
// tiles of 128, A and B, that take turns: while the tensor cores work for one,
// the softmax of the other runs.  Roles (sixteen warps, registers moved to the
// softmax's):
//   0-3, 4-7  softmax of A and of B, one row a thread; also its queries, the
//             rescaling of its accumulator and its output
//   8-11      V: codes into the 16-bit operand, from and to shared memory (and
//             K's into 8-bit ones, where they are E2M1)
//   12        issuing MMAs
//   13        all codes, by TMA
//   14        all scales
// For each unit of keys, S = Q K^T goes to tensor memory, its softmax weights P
// overwrite it there, and O += P V reads P from tensor memory.
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
#include <cuda.h>
#include <cudaTypedefs.h>
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
constexpr int kMinUnits = 2;
constexpr int kStages = 3;    // of K and of V
constexpr int kRawStages = 2; // of codes on their way to V
constexpr int kMetaRing = 8;  // more units than can be between their scales' arrival and their softmax
// Registers a thread by warpgroup; the launch's 128 x 4 are shared out.
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 168, kValueRegs = 112, kIssueRegs = 64;
static_assert(2 * kSoftmaxRegs + kValueRegs + kIssueRegs <= 4 * kLaunchRegs, "setmaxnreg would wait for ever");

// What the softmax and the MMA issuer need to know of a unit.
struct UnitMeta {
  int v_exp;  // exponent of its largest V scale
  int wide;   // V and P in bf16
  int lo, hi; // the keys that some row sees, counted from the unit's first
};

template <int D>
struct Shape {
  // Keys of a unit.  Tensor memory has 512 columns: two S (one a key), two O
  // (one an element) and the scales' 28; with 128 elements that leaves 96 keys in
  // steps of 32 columns.
  static constexpr int kUnit = D == 128 ? 96 : 128;
  static constexpr uint32_t kQTile = 128 * D;                // one 8-bit operand
  static constexpr uint32_t kKStage = kUnit * D;
  static constexpr uint32_t kVPanel = kUnit * 128;           // 64 16-bit elements of each key
  static constexpr uint32_t kVStage = kVPanel * (D / 64);
  static constexpr uint32_t kQ = 0;                          // A hi, A lo, B hi, B lo
  static constexpr uint32_t kK = 4 * kQTile;
  static constexpr uint32_t kV = kK + kStages * kKStage;
  // codes as they come: V's, and K's where they are E2M1
  static constexpr uint32_t kRaw = kV + kStages * kVStage;
  static constexpr uint32_t kRawStage = kUnit * D;
  static constexpr uint32_t kBytes = kRaw + kRawStages * kRawStage;
  static_assert(kKStage % 1024 == 0 && kVPanel % 1024 == 0, "swizzle atoms");
  // tensor memory columns
  static constexpr uint32_t kS = 0, kSNext = kUnit;
  static constexpr uint32_t kO = 256;                        // A, then B D on
  static constexpr uint32_t kScales = D == 128 ? 192 : 384;  // Q: A hi, A lo, B hi, B lo, then K's stages, four each
};
constexpr uint32_t kTmemColumns = 512;

struct Shared {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], drain;
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint32_t tmem;
  volatile int failed;
  int last[2];
  UnitMeta meta[kMetaRing];
  uint32_t q_scale[2][128];  // a row's scale bytes
  alignas(128) uint32_t k_scale[kStages][32][4];  // keys 32 j + lane, by lane
  uint32_t v_scale[kRawStages][128];
  int64_t units[kAttnScan];
};

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

// A wait that runs out sets the status word and makes every later wait of the
// CTA give up at once.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1; !mbar_try_wait(b, parity); ++n) {
    if (n & 15u) continue;
    if (sh.failed) return false;
    if (globaltimer_ns() - t0 > a.wait_limit_ns) {
      sh.failed = 1;
      set_status(a.status, MX_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void named_barrier(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
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
  if (a.lse) a.lse[oh] = L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
}
// Four elements of a row of a part: the same elements of all rows side by side.
template <int D>
__device__ __forceinline__ float4* part_at(const AttnArgs& a, int slot, int d4, int row) {
  return reinterpret_cast<float4*>(a.part_o) + (static_cast<int64_t>(slot) * (D / 4) + d4) * kRows + row;
}

// A tile's queries as two MXFP8 operands and their scales, by the 128 threads of
// its softmax: eight elements a lane at a time, four lanes a block.  Not inlined
// (nor is join_parts): once a segment, and it would push the unit loops out of
// the instruction cache.
template <int D>
__device__ __noinline__ void load_queries(const AttnArgs& a, Shared& sh, uint8_t* base, int x, int q0, int head, int row0,
                                          int rows) {
  using Sh = Shape<D>;
  constexpr uint32_t tmem = 0;
  const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(threadIdx.x & 96) << 16;
        constexpr int kPieces = D / 8;
              uint8_t* hi_base = base + Sh::kQ + 2 * x * Sh::kQTile;
#pragma unroll 2
        for (int i = row; i < 128 * kPieces; i += 128) {
          const int r = i / kPieces, p = i - r * kPieces;
          const int R = row0 + r;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (R < rows) {
            const int tok = R / a.group;
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                     static_cast<int64_t>(q0 + tok) * a.q_stride +
                                                     static_cast<int64_t>(head * a.group + (R - tok * a.group)) * D) + p);
          }
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t amax = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) amax = max(amax, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // the block's largest element lands in [2^7, 2^8): hi's rounding error
          // is then at most 2^3 and 2^5 times it stays below E4M3's 448
          const int s = max(static_cast<int>(amax >> 7) - 127 - 7, -122);
          const float down = pow2_neg(s);
          uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x0 = __uint_as_float(w[k] << 16) * down, x1 = __uint_as_float(w[k] & 0xFFFF0000u) * down;
            const uint32_t h = enc_e4m3x2(x0, x1);
            const uint32_t back = f16x2_of_e4m3x2(h);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
            hi[k >> 1] |= h << ((k & 1) * 16);
            lo[k >> 1] |= enc_e4m3x2((x0 - f.x) * 32.0f, (x1 - f.y) * 32.0f) << ((k & 1) * 16);
          }
          const uint32_t at = D == 128 ? r * 128 + (((p >> 1) ^ (r & 7)) << 4) + (p & 1) * 8
                                       : r * 64 + (((p >> 1) ^ ((r >> 1) & 3)) << 4) + (p & 1) * 8;
          *reinterpret_cast<uint2*>(hi_base + at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(hi_base + Sh::kQTile + at) = make_uint2(lo[0], lo[1]);
          if ((p & 3) == 0) reinterpret_cast<uint8_t*>(&sh.q_scale[x][r])[p >> 2] = static_cast<uint8_t>(s + 127);
        }
        fence_proxy_async_shared();
        named_barrier(1 + x);
        // scales: row 32 j + lane in column j, the same in every lane quarter
        const uint32_t col = tmem + lanes + Sh::kScales + 8u * x;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = sh.q_scale[x][32 * j + lane];
        tmem_st_32x32b_x4(col, w[0], w[1], w[2], w[3]);
        constexpr uint32_t kFive = D == 128 ? 0x05050505u : 0x0505u;
        tmem_st_32x32b_x4(col + 4, w[0] - kFive, w[1] - kFive, w[2] - kFive, w[3] - kFive);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&sh.q_full[x]));
}

// A row of a split segment from its parts, in key order.
template <int D>
__device__ __noinline__ void join_parts(const AttnArgs& a, AttnParts p, int row, int64_t oh) {
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
    put<D>(a, oh, c, f, L > 0.0f ? 1.0f / L : 0.0f);
  }
  put_lse(a, oh, M, L);
}

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads, 1) k_attn_chunk(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                                                              const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<D>;
  constexpr int kUnit = Sh::kUnit;
  using Cursor = AttnCursor<kRows, kUnit>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same for the warp, and known to be
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 128);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 128);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), E2M1 ? 129 : 2);  // scales, and codes by TMA or by V's warps
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), 128);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(smem_u32(&sh.raw_full[i]), 2);  // scales and codes
      mbar_init(smem_u32(&sh.raw_empty[i]), 128);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.failed = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&sh.tmem), kTmemColumns);
    tmem_relinquish();
  }
  const AttnShare share = attn_share<kRows, kUnit, kThreads, true>(a, sh.units);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all of tensor memory is this CTA's
  int64_t u = share.u;
  Cursor cur;
  if (u < share.end) cur.template start<true>(a, share);
  // Where a unit lies, its 16-key groups by lane: looked up one unit before it
  // is needed, and the page id left alone until then.
  struct Place {
    int page, head;  // as the table has it
    int offset;      // the group's first place in the page, or -1: no row sees it
    int lo, hi;      // the keys to read, counted from the unit's first
  };
  auto look_up = [&](const Cursor& c, int group) {
    Place p;
    const int key = c.t.first + c.place * kUnit + 16 * group;
    const int entry = key / a.page_size;
    p.lo = c.t.lo - (key - 16 * group);
    p.hi = c.t.hi - (key - 16 * group);
    p.head = c.head;
    const bool seen = group < kUnit / 16 && 16 * group < p.hi && 16 * group + 16 > p.lo;
    p.offset = seen ? key - entry * a.page_size : -1;
    p.page = __ldg(a.block_table + static_cast<int64_t>(c.b) * a.max_pages + (seen ? entry : 0));
    return p;
  };
  // The group's first cache row, or -1 where it is not there.
  auto group_row = [&](const Place& p) {
    if (p.offset < 0) return -1;
    if (p.page < 0 || p.page >= a.num_pages) {
      set_status(a.status, MX_ERR_DEVICE_ARG);
      return -1;
    }
    return (p.page * a.n_kv_heads + p.head) * a.page_size + p.offset;
  };

  if (warp < 8) {
    // ================================================================ softmax
    take_registers<kSoftmaxRegs>();
    const int x = warp >> 2;                       // tile A or B
    const int row = tid & 127;                     // the thread's row of it
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + Sh::kS + Sh::kSNext * x, o_col = tmem + lanes + Sh::kO + D * static_cast<uint32_t>(x);
    const int n_heads = a.n_kv_heads * a.group;
    uint32_t unit = 0, s_phase = 0, o_phase = 0;
    bool ok = true;

    sh.q_scale[x][row] = 0u;
    named_barrier(1 + x);
    auto queries_of = [&](const Cursor& c) {
      const int rows = c.s.n * a.group, row0 = c.tile * kRows + 128 * x;
      if (row0 < rows) load_queries<D>(a, sh, base, x, c.s.q0, c.head, row0, rows);
    };
    if (u < share.end) queries_of(cur);
    while (u < share.end && cur.b < a.n_seqs) {
      const int take = static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), share.end - u));
      const int rows = cur.s.n * a.group;
      const int row0 = cur.tile * kRows + 128 * x;
      Cursor ahead;
      auto to_next = [&]() {  // and its queries
        ahead = cur;
        if (u + take >= share.end) return;
        ahead.next(a);
        if (ahead.b < a.n_seqs) queries_of(ahead);
      };
      if (row0 < rows) {
        const int R = row0 + row;
        const bool valid = R < rows;
        const int tok = valid ? R / a.group : 0;
        const int at = cur.s.kv - cur.s.n + tok;
        // rows past the last see everything: their queries are zero
        const int hi = !valid ? INT_MAX : a.causal ? min(cur.s.kv, max(at + 1, 0)) : cur.s.kv;
        const int lo = valid && a.window > 0 ? max(at - a.window + 1, 0) : 0;
        const int all_hi = __reduce_min_sync(0xffffffffu, hi), all_lo = __reduce_max_sync(0xffffffffu, lo);
        const bool warp_valid = row0 + 32 * (warp & 3) < rows;
        const float scale = a.scale_log2;
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (int j = 0; j < take; ++j) {
          if (ok) ok = wait(sh, &sh.s_full[x], s_phase, a);
          s_phase ^= 1u;
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          if (ok && warp_valid) {
            const UnitMeta meta = sh.meta[(unit + j) % kMetaRing];
            const int key0 = cur.t.first + (cur.place + j) * kUnit;
            if (key0 + kUnit > all_hi || key0 < all_lo) {
              const int c_hi = hi - key0, c_lo = lo - key0;  // the columns that the row sees
#pragma unroll 1
              for (int c = 0; c < kUnit; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(s_col + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (c + i >= c_hi || c + i < c_lo) v[i] = 0xFF800000u;
                tmem_st_32x32b_x16(s_col + c, v);
              }
              tmem_st_wait();
            }
            // The code that runs for every unit is kept short: the warps' roles
            // differ, and together they have to fit the instruction cache.
            uint32_t v[kUnit];
            tmem_load<kUnit>(s_col, v);
            tmem_ld_wait();
            float t4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t4[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[4 + k]));
#pragma unroll
            for (int i = 8; i < kUnit; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) t4[k] = fmaxf(t4[k], fmaxf(__uint_as_float(v[i + k]), __uint_as_float(v[i + 4 + k])));
            }
            const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            const float e = static_cast<float>(meta.v_exp);
            const float joint = fmaf(top, scale, e);
            if (__any_sync(0xffffffffu, joint > m + 8.0f)) {
              const float to = fmaxf(m, joint);
              const float f = to == -INFINITY ? 1.0f : exp2_approx(m - to);
              // O holds something but zeros once a row has seen a key; the MMA
              // that S waited for was issued behind the last one that writes O
              const bool rescale = __any_sync(0xffffffffu, m != -INFINITY);
              m = to;
              l *= f;
              if (rescale) {
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
            }
            const float off = m == -INFINITY ? 0.0f : e - m;
            const float2 scale2 = make_float2(scale, scale), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            if (__builtin_expect(meta.wide == 0, 1)) {
#pragma unroll
              for (int i = 0; i < kUnit; i += 2) {
                const float2 z = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), scale2, off2);
                const float2 w = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], w);
                v[i / 2] = pack_f16(w.x, w.y);
              }
#pragma unroll
              for (int c = 0; c < kUnit / 2; c += 16) tmem_st_32x32b_x16(s_col + c, reinterpret_cast<uint32_t(&)[16]>(v[c]));
            } else {
#pragma unroll 1
              for (int c = 0; c < kUnit; c += 32) {
                uint32_t z[32], p[16];
                tmem_ld_32x32b_x32(s_col + c, z);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const float2 y = fma2(make_float2(__uint_as_float(z[i]), __uint_as_float(z[i + 1])), scale2, off2);
                  const float2 w = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                  sum[0] = add2(sum[0], w);
                  p[i / 2] = pack_bf16(w.x, w.y);
                }
                tmem_st_32x32b_x16(s_col + c / 2, p);  // behind the columns read so far
              }
            }
            const float2 all = add2(sum[0], sum[1]);
            l = fmaf(all.x + all.y, __uint_as_float(static_cast<uint32_t>(127 - meta.v_exp) << 23), l);
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&sh.p_full[x]));
        }
        // the last scores are done: the next segment's queries may come
        to_next();

        // ---------------------------------------------------------------- output
        if (ok) ok = wait(sh, &sh.o_full[x], o_phase, a);
        o_phase ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const bool whole = take == cur.t.units;
        const int64_t oh = static_cast<int64_t>(cur.s.q0 + tok) * n_heads + cur.head * a.group + (R - tok * a.group);
        const int slot = attn_slot(blockIdx.x, cur.place == 0);
        if (ok && warp_valid) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 2
          for (int c = 0; c < D; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(o_col + c, v);
            tmem_ld_wait();
            float f[16];
            // a row without a visible key never had its accumulator's weights defined
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = l > 0.0f ? __uint_as_float(v[i]) : 0.0f;
            if (valid && whole) {
              put<D>(a, oh, c, f, inv);
            } else if (valid) {
#pragma unroll
              for (int i = 0; i < 4; ++i) *part_at<D>(a, slot, c / 4 + i, 128 * x + row) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
            __syncwarp();
          }
          if (valid) {
            if (whole) put_lse(a, oh, m, l);
            else a.part_ml[slot * kRows + 128 * x + row] = make_float2(m, l);
          }
        }
        if (!whole) {
          const AttnParts parts = attn_parts(share, u - cur.place, cur.t.units);
          // also after a wait that ran out: the counters are zero for the next call
          __threadfence();
          named_barrier(1 + x);
          unsigned* counter = &a.arrived[2 * parts.first + x];
          if (row == 0) {
            sh.last[x] = atomicAdd(counter, 1u) == static_cast<unsigned>(parts.parts - 1);
            if (sh.last[x]) *counter = 0u;
          }
          named_barrier(1 + x);
          if (sh.last[x] && ok && valid) {
            __threadfence();
            join_parts<D>(a, parts, 128 * x + row, oh);
          }
        }
      } else {
        to_next();  // this segment has no tile B
      }
      unit += take;
      u += take;
      cur = ahead;
    }
  } else if (warp < 12) {
    // ================================================================ V, and K's scales
    give_registers<kValueRegs>();
    constexpr int kShares = D / 16;            // lanes of a key: sixteen elements each
    constexpr int kKeysPerIt = 128 / kShares;  // over the four warps
    constexpr int kRowBytes = E2M1 ? D / 2 : D;
    constexpr int kPieceBytes = kRowBytes / kShares;
    const int dw = warp - 8;
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
    const int n = static_cast<int>(share.end - share.u);
    Ring<kStages> ring;
    Ring<kRawStages> raw;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      bool ok = wait(sh, &sh.raw_full[raw.stage], raw.phase, a);
      if (E2M1 && ok) ok = wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
      if (ok) ok = wait(sh, &sh.v_empty[ring.stage], ring.phase ^ 1u, a);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const UnitMeta meta = sh.meta[static_cast<uint32_t>(i) % kMetaRing];
      const uint8_t* codes = base + Sh::kRaw + raw.stage * Sh::kRawStage + r0 * kRowBytes + part * kPieceBytes;
      const uint8_t* scales = reinterpret_cast<const uint8_t*>(&sh.v_scale[raw.stage][r0]) + part / 2;
      uint8_t* v_to = base + Sh::kV + ring.stage * Sh::kVStage;
      const bool cut = meta.lo > 0 || meta.hi < kUnit;
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
        mbar_arrive(smem_u32(&sh.k_full[ring.stage]));
      }
      if (__builtin_expect(meta.wide, 0)) {
#pragma unroll 1
        for (int r = 0; r < kUnit; r += kKeysPerIt) {
          Codes<E2M1> v;
          v.load(codes + r * kRowBytes);
          if (cut && (r + r0 < meta.lo || r + r0 >= meta.hi)) v.clear();
          const uint32_t f = bf16_pow2x2_112(min(scales[r * 4] - 127 - meta.v_exp, 15));
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(bf16x2_of_f16x2(v.pair(e)), f);
          *reinterpret_cast<uint4*>(v_to + v_at0 + r * 128) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(v_to + v_at1 + r * 128) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
#pragma unroll 2
        for (int r = 0; r < kUnit; r += kKeysPerIt) {
          Codes<E2M1> v;
          v.load(codes + r * kRowBytes);
          if (cut && (r + r0 < meta.lo || r + r0 >= meta.hi)) v.clear();
          const uint32_t f = f16_pow2x2(min(scales[r * 4] - 127 - meta.v_exp, 15));
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = mul_f16x2(v.pair(e), f);
          *reinterpret_cast<uint4*>(v_to + v_at0 + r * 128) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(v_to + v_at1 + r * 128) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      fence_proxy_async_shared();
      mbar_arrive(smem_u32(&sh.v_full[ring.stage]));
      mbar_arrive(smem_u32(&sh.raw_empty[raw.stage]));
      ring.next();
      raw.next();
    }
  } else {
    give_registers<kIssueRegs>();
    if (warp == 12) {
      if (elect_one()) {
      // ================================================================ MMAs
      // V is MN-major: 64-element panels along N lie kVPanel apart (leading
      // offset), eight-key groups 1024 bytes (stride)
      const uint32_t q_lo = desc_lo_sw128(smem_u32(base + Sh::kQ)), k_lo = desc_lo_sw128(smem_u32(base + Sh::kK));
      const uint32_t v_lo = ((smem_u32(base + Sh::kV) >> 4) & 0x3FFFu) | ((Sh::kVPanel >> 4) << 16);
      constexpr uint32_t kQkHi = D == 128 ? kDescHiSw128 : kDescHiSw64;
      uint32_t q_phase = 0, p_phase = 0;
      bool ok = true;
      auto scores = [&](uint32_t x, uint32_t stage) {
        const uint32_t d = tmem + Sh::kS + Sh::kSNext * x;
        const uint32_t q_sf = tmem + Sh::kScales + 8u * x, k_sf = tmem + Sh::kScales + 16u + 4u * stage;
        const uint32_t q = q_lo + ((2 * x * Sh::kQTile) >> 4), k = k_lo + ((stage * Sh::kKStage) >> 4);
#pragma unroll
        for (uint32_t part = 0; part < 2; ++part) {
#pragma unroll
          for (uint32_t b = 0; b < D / 32; ++b)
            mma_mxf8f6f4_lo(d, q + ((part * Sh::kQTile) >> 4) + 2u * b, k + 2u * b, kQkHi,
                            idesc_mx(kFmtE4M3, kFmtE4M3, 128, kUnit, b, b), q_sf + 4u * part, k_sf, (part | b) != 0);
        }
        mma_commit(smem_u32(&sh.s_full[x]));
      };
      auto values = [&](uint32_t x, uint32_t stage, uint32_t idesc, bool first) {
#pragma unroll
        for (uint32_t k = 0; k < kUnit / 16; ++k)
          mma_f16_ts(tmem + Sh::kO + D * x, tmem + Sh::kS + Sh::kSNext * x + 8u * k,
                     v_lo + ((stage * Sh::kVStage + k * 2048u) >> 4), kDescHiSw128, idesc, !first || k != 0);
      };
      uint32_t unit = 0;
      Ring<kStages> kr, vr;  // the next stage to take
      while (ok && u < share.end && cur.b < a.n_seqs) {
        const int take = static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), share.end - u));
        const uint32_t tiles = cur.s.n * a.group - cur.tile * kRows > 128 ? 2 : 1;
        for (uint32_t x = 0; x < tiles && ok; ++x) ok = wait(sh, &sh.q_full[x], (q_phase >> x) & 1u, a);
        q_phase ^= tiles == 2 ? 3u : 1u;
        // step j: O += P V of unit j, then S of unit j + 1, tile by tile
#pragma unroll 1
        for (int j = -1; j < take && ok; ++j) {
          const bool more = j + 1 < take;
          uint32_t idesc = 0;
          if (j >= 0) {
            ok = wait(sh, &sh.v_full[vr.stage], vr.phase, a);
            if (!ok) break;
            idesc = idesc_f16(sh.meta[unit % kMetaRing].wide != 0, true, 128, D);
            ++unit;
          }
#pragma unroll 1
          for (uint32_t x = 0; x < tiles; ++x) {
            if (j >= 0) {
              ok = wait(sh, &sh.p_full[x], (p_phase >> x) & 1u, a);
              if (!ok) break;
              tc_fence_after();
              values(x, vr.stage, idesc, j == 0);
            }
            if (more) {
              // P lies in S: these MMAs are issued behind the ones that read it
              if (x == 0) {
                ok = wait(sh, &sh.k_full[kr.stage], kr.phase, a);
                if (!ok) break;
                tc_fence_after();
                tmem_copy_scales(tmem + Sh::kScales + 16u + 4u * kr.stage, smem_u32(&sh.k_scale[kr.stage][0][0]));
              }
              scores(x, kr.stage);
            } else {
              mma_commit(smem_u32(&sh.o_full[x]));
            }
          }
          if (!ok) break;
          if (j >= 0) {
            p_phase ^= tiles == 2 ? 3u : 1u;
            mma_commit(smem_u32(&sh.v_empty[vr.stage]));
            vr.next();
          }
          if (more) {
            mma_commit(smem_u32(&sh.k_empty[kr.stage]));
            kr.next();
          }
        }
        u += take;
        if (ok && u < share.end) cur.next(a);
      }
      // every MMA issued has completed before tensor memory is released
      mma_commit(smem_u32(&sh.drain));
      mbar_wait(smem_u32(&sh.drain), 0, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 13) {
      // ================================================================ codes
      // Sixteen keys a TMA box, each by its own lane (K's from lane 0, V's from
      // lane 16 on); a group that is not there is read past the table's end,
      // which fills zeros.
      const int n = static_cast<int>(share.end - share.u);
      const int none = a.num_pages * a.n_kv_heads * a.page_size;
      constexpr uint32_t kCodeBytes = E2M1 ? Sh::kRawStage / 2 : Sh::kRawStage;  // of K or V
      constexpr uint32_t kGroupBytes = kCodeBytes / (kUnit / 16);
      int left = n > 0 ? static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), static_cast<int64_t>(n))) : 0;
      Ring<kStages> ring;
      Ring<kRawStages> raw;
      bool ok = true;
      int issued = 0;
      if (lane < 2) prefetch_tensormap(lane == 0 ? &k_map : &v_map);
      const int group = lane & 15;
      Place at{};
#pragma unroll 1
      for (int i = -1; i < n; ++i) {
        const int found = i >= 0 ? group_row(at) : -1;
        const int row = found < 0 ? none : found;
        if (i + 1 < n) {
          if (i >= 0) {
            if (--left == 0) {
              cur.next(a);
              left = cur.t.units;
            } else {
              ++cur.place;
            }
          }
          at = look_up(cur, group);
        }
        if (i < 0) continue;
        if (!E2M1) ok = wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
        if (ok) ok = wait(sh, &sh.raw_empty[raw.stage], raw.phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t k_bar = smem_u32(E2M1 ? &sh.raw_full[raw.stage] : &sh.k_full[ring.stage]);
        const uint32_t v_bar = smem_u32(&sh.raw_full[raw.stage]);
        if (lane == 0) {
          mbar_arrive_expect_tx(v_bar, E2M1 ? 2 * kCodeBytes : kCodeBytes);
          if (!E2M1) mbar_arrive_expect_tx(k_bar, kCodeBytes);
        }
        __syncwarp();
        if (group < kUnit / 16) {
          const uint32_t v_to = smem_u32(base + Sh::kRaw + raw.stage * Sh::kRawStage) + group * kGroupBytes;
          const uint32_t k_to = E2M1 ? v_to + kCodeBytes : smem_u32(base + Sh::kK + ring.stage * Sh::kKStage) + group * kGroupBytes;
          if (lane < 16) tma_load_2d(k_to, &k_map, 0, row, k_bar);
          else tma_load_2d(v_to, &v_map, 0, row, v_bar);
        }
        __syncwarp();
        ++issued;
        ring.next();
        raw.next();
      }
      // the last fills have landed before the CTA exits, also where a wait of
      // the others ran out
      for (int i = issued > kRawStages ? issued - kRawStages : 0; i < issued; ++i)
        mbar_wait(smem_u32(&sh.raw_full[i % kRawStages]), (i / kRawStages) & 1u, 100000000ull);
      for (int i = issued > kStages ? issued - kStages : 0; i < issued && !E2M1; ++i)
        mbar_wait(smem_u32(&sh.k_full[i % kStages]), (i / kStages) & 1u, 100000000ull);
      __syncwarp();
    } else if (warp == 14) {
      // ================================================================ scales
      constexpr int kWords = kUnit / 32, kBlocks = D / 32;
      const int n = static_cast<int>(share.end - share.u);
      int left = n > 0 ? static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), static_cast<int64_t>(n))) : 0;
      Ring<kStages> ring;
      Ring<kRawStages> raw;
      auto scale_word = [&](const uint8_t* p, int64_t row) -> uint32_t {
        if constexpr (kBlocks == 4) return __ldg(reinterpret_cast<const uint32_t*>(p) + row);
        else return __ldg(reinterpret_cast<const uint16_t*>(p) + row);
      };
      struct Unit {
        uint32_t ks[kWords], vs[kWords];  // keys 32 j + lane: a row's scale bytes
        uint32_t gone;                    // bit g: 16-key group g is not there
        int lo, hi;
      };
      Place at{};
      Unit now, then;
      // In each turn one unit is looked up, the one before it loaded, and the one
      // before that, whose loads have had a turn to arrive, passed on.  What no
      // row sees is read as whatever lies in its place (the table's first rows
      // where there is none) and left out later: choosing between a load's
      // result and a constant would wait for the load.
#pragma unroll 1
      for (int i = -2; i < n; ++i) {
        if (i >= 0) now = then;
        if (i >= -1 && i + 1 < n) {
          const int row = group_row(at);
          const int first_row = max(row, 0);
          then.gone = __ballot_sync(0xffffffffu, lane < kUnit / 16 && row < 0);
          then.lo = at.lo;
          then.hi = at.hi;
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const int64_t to = __shfl_sync(0xffffffffu, first_row, 2 * j + lane / 16) + lane % 16;
            then.ks[j] = scale_word(a.k_scales, to);
            then.vs[j] = scale_word(a.v_scales, to);
          }
        }
        if (i + 2 < n) {
          if (i > -2) {
            if (--left == 0) {
              cur.next(a);
              left = cur.t.units;
            } else {
              ++cur.place;
            }
          }
          at = look_up(cur, lane);
        }
        if (i < 0) continue;
        bool ok = wait(sh, &sh.k_empty[ring.stage], ring.phase ^ 1u, a);
        if (ok) ok = wait(sh, &sh.raw_empty[raw.stage], raw.phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        *reinterpret_cast<uint4*>(&sh.k_scale[ring.stage][lane][0]) =
            make_uint4(now.ks[0], now.ks[1], now.ks[2], kWords == 4 ? now.ks[kWords - 1] : 0x7F7F7F7Fu);
        fence_proxy_async_shared();
        // V's largest scale, and the smallest of a block that is not zero
        uint32_t top = 0, low = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const int r = 32 * j + lane;
          const uint32_t w = r >= now.lo && r < now.hi && !(now.gone >> (r / 16) & 1u) ? now.vs[j] : 0u;
          sh.v_scale[raw.stage][r] = w;
          top = __vmaxu4(top, w);
          low = __vminu4(low, w | __vcmpeq4(w, 0u));
        }
        top = max(max(top & 0xFFu, (top >> 8) & 0xFFu), max((top >> 16) & 0xFFu, top >> 24));
        low = min(min(low & 0xFFu, (low >> 8) & 0xFFu), min((low >> 16) & 0xFFu, low >> 24));
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) {
          UnitMeta meta;
          meta.v_exp = min(max(static_cast<int>(top) - 127, -100), 126);
          meta.wide = meta.v_exp - (static_cast<int>(low) - 127) > 15;
          meta.lo = now.lo;
          meta.hi = now.hi;
          sh.meta[static_cast<uint32_t>(i) % kMetaRing] = meta;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.k_full[ring.stage]));
          mbar_arrive(smem_u32(&sh.raw_full[raw.stage]));
        }
        __syncwarp();
        ring.next();
        raw.next();
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(sh.tmem, kTmemColumns);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
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
    // the register split counts on the launch's 128 a thread
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, k_attn_chunk<D, E2M1>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(k_attn_chunk<D, E2M1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  // K's E4M3 rows are an MMA operand as they are, swizzled on their way; the
  // codes that pass through V's warps keep their order
  auto encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap k_map, v_map;
  const cuuint64_t row = E2M1 ? D / 2 : D;
  cuuint64_t dims[2] = {row, static_cast<cuuint64_t>(a.num_pages) * a.n_kv_heads * a.page_size}, strides[1] = {row};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(row), 16}, es[2] = {1, 1};
  const CUtensorMapSwizzle k_swizzle =
      E2M1 ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (encode(&k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.k_codes), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, k_swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      encode(&v_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.v_codes), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
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
