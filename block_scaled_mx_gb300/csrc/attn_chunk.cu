// Attention of chunks of new tokens over the paged MX cache on the tensor
// cores: tcgen05 MMAs with the accumulators in tensor memory, bound by the
// MMAs (4 * head_dim flops for each visible (row, key) pair).
//
// A tile is 256 rows (new tokens x the query heads of one KV head) as two MMA
// tiles of 128, A and B, that take turns: while the tensor cores work for one,
// the softmax of the other runs.  Keys come in units of 128.  Roles (13 warps):
//   0-3, 4-7  softmax of A and of B, one row a thread; also its queries, the
//             rescaling of its accumulator and its output
//   8-11      reading the cache: codes and scales through registers into the
//             16-bit operands in shared memory (two stages of K and of V)
//   12        issuing MMAs
// For each unit, S = Q K^T goes to tensor memory, its softmax weights P
// overwrite it there, and O += P V reads P from tensor memory.
//
// Arithmetic.  Q and K are bf16: every code times its scale is exact there,
// relative to the unit's largest K scale, which multiplies the score in fp32.
// V is exact in f16 relative to the unit's largest V scale e as long as the
// unit's scales lie within 2^15; P is then rounded to f16 (2^-11).  A unit with
// a wider spread takes bf16 for both (V exact, P 2^-8).  As in the few-rows
// kernel e joins the softmax's exponent: P = 2^(x + e - M) with M the running
// maximum of x + e, and the sum adds (sum of P) 2^-e.  M moves only when it
// would grow by more than 2^8, so O is seldom rescaled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "attn.cuh"
#include "kv.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int kRows = 256;
constexpr int kUnit = 128;
constexpr int kThreads = 416;
constexpr int kMaxCtas = 152;
constexpr int kMinUnits = 2;
constexpr uint32_t kPanel = 128 * 128;  // 128 rows of 64 16-bit elements
constexpr int kMetaRing = 4;

// What the softmax and the MMA issuer need to know of a unit.
struct UnitMeta {
  float k_scale;  // 2^e of the unit's largest K scale
  int v_exp;      // e of its largest V scale
  int wide;       // V and P in bf16
};

template <int D>
struct Layout {
  static constexpr uint32_t kTile = D / 64 * kPanel;  // one 128-row operand
  static constexpr uint32_t kQ = 0;                   // A, B
  static constexpr uint32_t kK = 2 * kTile;           // two stages
  static constexpr uint32_t kV = 4 * kTile;
  static constexpr uint32_t kBytes = 6 * kTile;
  // tensor memory columns
  static constexpr uint32_t kS = 0;    // A, then B 128 on
  static constexpr uint32_t kO = 256;  // A, then B D on
};
constexpr uint32_t kTmemColumns = 512;

struct Shared {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], drain;
  uint32_t tmem;
  volatile int failed;
  int last[2];
  UnitMeta meta[kMetaRing];
  int scale_max[2][4][3];  // by parity and warp: largest K scale, largest and smallest V scale
  int64_t units[kAttnScan];
};

// A wait that runs out sets the status word and makes every later wait of the
// CTA give up at once.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(b, parity)) {
    if (sh.failed) return false;
    if (globaltimer_ns() - t0 > a.wait_limit_ns) {
      sh.failed = 1;
      set_status(a.status, MX_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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

// Sixteen codes of one key, a lane's share.
template <bool E2M1>
struct Codes {
  uint32_t w[E2M1 ? 2 : 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (E2M1) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (E2M1 ? 2 : 4); ++i) w[i] = 0u;
  }
  // elements 2i, 2i + 1
  __device__ __forceinline__ uint32_t pair(int i) const {
    if constexpr (E2M1) return f16x2_of_e2m1x2((w[i / 4] >> (8 * (i % 4))) & 0xFFu);
    else return f16x2_of_e4m3x2((w[i / 2] >> (16 * (i % 2))) & 0xFFFFu);
  }
};

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads, 1) k_attn_chunk(const AttnArgs a) {
  using L = Layout<D>;
  using Cursor = AttnCursor<kRows, kUnit>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), 128);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 128);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
      mbar_init(smem_u32(&sh.k_full[i]), 128);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), 128);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
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
  const uint32_t tmem = sh.tmem;
  int64_t u = share.u;
  Cursor cur;
  if (u < share.end) cur.template start<true>(a, share);
  uint32_t unit = 0;  // units so far, over all segments: stages and phases

  if (warp < 8) {
    // ================================================================ softmax
    const int x = warp >> 2;                       // tile A or B
    const int row = tid & 127;                     // the thread's row of it
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + L::kS + 128u * x, o_col = tmem + lanes + L::kO + D * static_cast<uint32_t>(x);
    const int n_heads = a.n_kv_heads * a.group;
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    while (u < share.end && cur.b < a.n_seqs) {
      const int take = static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), share.end - u));
      const int rows = cur.s.n * a.group;
      const int row0 = cur.tile * kRows + 128 * x;
      if (row0 < rows) {
        // queries: sixteen-byte pieces, D / 8 of them a row, swizzled
        constexpr int kPieces = D / 8;
#pragma unroll 4
        for (int i = row; i < 128 * kPieces; i += 128) {
          const int r = i / kPieces, p = i - r * kPieces;
          const int R = row0 + r;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (R < rows) {
            const int tok = R / a.group;
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                     static_cast<int64_t>(cur.s.q0 + tok) * a.q_stride +
                                                     static_cast<int64_t>(cur.head * a.group + (R - tok * a.group)) * D) + p);
          }
          *reinterpret_cast<uint4*>(base + L::kQ + x * L::kTile + (p / 8) * kPanel + r * 128 + (((p & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_shared();
        mbar_arrive(smem_u32(&sh.q_full[x]));

        const int R = row0 + row;
        const bool valid = R < rows;
        const int tok = valid ? R / a.group : 0;
        const int at = cur.s.kv - cur.s.n + tok;
        // rows past the last see everything: their queries are zero
        const int hi = !valid ? INT_MAX : a.causal ? min(cur.s.kv, max(at + 1, 0)) : cur.s.kv;
        const int lo = valid && a.window > 0 ? max(at - a.window + 1, 0) : 0;
        const int all_hi = __reduce_min_sync(0xffffffffu, hi), all_lo = __reduce_max_sync(0xffffffffu, lo);
        const bool warp_valid = row0 + 32 * (warp & 3) < rows;
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; j < take; ++j) {
          if (ok) ok = wait(sh, &sh.s_full[x], s_phase, a);
          s_phase ^= 1u;
          tc_fence_after();
          ok = __all_sync(0xffffffffu, ok);
          if (ok && warp_valid) {
            const UnitMeta meta = sh.meta[(unit + j) % kMetaRing];
            const int key0 = cur.t.first + (cur.place + j) * kUnit;
            const bool masked = key0 + kUnit > all_hi || key0 < all_lo;
            const float scale = a.scale_log2 * meta.k_scale;
            // the columns that the row sees
            const int c_hi = hi - key0, c_lo = lo - key0;
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < kUnit; c += 32) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(s_col + c, v);
              tmem_ld_wait();
              if (masked) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (c + i < c_hi && c + i >= c_lo) top = fmaxf(top, __uint_as_float(v[i]));
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(v[i]));
              }
            }
            const float e = static_cast<float>(meta.v_exp);
            const float joint = fmaf(top, scale, e);
            if (__any_sync(0xffffffffu, joint > m + 8.0f)) {
              const float to = fmaxf(m, joint);
              const float f = to == -INFINITY ? 1.0f : exp2_approx(m - to);
              m = to;
              l *= f;
              if (j > 0) {  // the MMA that S waited for was issued behind the last one that writes O
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                  uint32_t v[32];
                  tmem_ld_32x32b_x32(o_col + c, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                  tmem_st_32x32b_x32(o_col + c, v);
                }
              }
            }
            const float off = m == -INFINITY ? 0.0f : e - m;
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < kUnit; c += 32) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(s_col + c, v);
              tmem_ld_wait();
              float w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i] = exp2_approx(fmaf(__uint_as_float(v[i]), scale, off));
              if (masked) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(c + i < c_hi && c + i >= c_lo)) w[i] = 0.0f;
              }
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                sum += w[2 * i] + w[2 * i + 1];
                p[i] = meta.wide ? pack_bf16(w[2 * i], w[2 * i + 1]) : pack_f16(w[2 * i], w[2 * i + 1]);
              }
              tmem_st_32x32b_x16(s_col + c / 2, p);  // behind the columns read so far
            }
            l = fmaf(sum, __uint_as_float(static_cast<uint32_t>(127 - meta.v_exp) << 23), l);
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(smem_u32(&sh.p_full[x]));
        }

        // ---------------------------------------------------------------- output
        if (ok) ok = wait(sh, &sh.o_full[x], o_phase, a);
        o_phase ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const bool whole = take == cur.t.units;
        const int64_t oh = static_cast<int64_t>(cur.s.q0 + tok) * n_heads + cur.head * a.group + (R - tok * a.group);
        // 32 finished elements of the row
        auto put = [&](int c, const float (&v)[32], float inv) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + oh * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
        };
        auto put_lse = [&](float M, float Lsum) {
          if (a.lse) a.lse[oh] = Lsum > 0.0f ? (M + log2f(Lsum)) * 0.69314718055994531f : -INFINITY;
        };
        const AttnParts parts = attn_parts(share, u - cur.place, cur.t.units);
        // a part's row lies with float4s of the same elements of all rows side by side
        auto part_at = [&](int slot, int d4) {
          return reinterpret_cast<float4*>(a.part_o) + (static_cast<int64_t>(slot) * (D / 4) + d4) * kRows + 128 * x + row;
        };
        const int slot = attn_slot(blockIdx.x, cur.place == 0);
        if (ok && warp_valid) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(o_col + c, v);
            tmem_ld_wait();
            float f[32];
            // a row without a visible key never had its accumulator's weights defined
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = l > 0.0f ? __uint_as_float(v[i]) : 0.0f;
            if (valid && whole) {
              put(c, f, l > 0.0f ? 1.0f / l : 0.0f);
            } else if (valid) {
#pragma unroll
              for (int i = 0; i < 8; ++i) *part_at(slot, c / 4 + i) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
            __syncwarp();
          }
          if (valid) {
            if (whole) put_lse(m, l);
            else a.part_ml[slot * kRows + 128 * x + row] = make_float2(m, l);
          }
        }
        if (!whole) {
          // also after a wait that ran out: the counters are zero for the next call
          __threadfence();
          named_barrier(1 + x, 128);
          unsigned* counter = &a.arrived[2 * parts.first + x];
          if (row == 0) {
            sh.last[x] = atomicAdd(counter, 1u) == static_cast<unsigned>(parts.parts - 1);
            if (sh.last[x]) *counter = 0u;
          }
          named_barrier(1 + x, 128);
          if (sh.last[x] && ok && valid) {
            __threadfence();
            float M = -INFINITY;
            for (int i = 0; i < parts.parts; ++i)
              M = fmaxf(M, __ldcg(&a.part_ml[attn_slot(parts.first + i, i == 0) * kRows + 128 * x + row]).x);
            float Lsum = 0.0f;
            for (int i = 0; i < parts.parts; ++i) {
              const float2 ml = __ldcg(&a.part_ml[attn_slot(parts.first + i, i == 0) * kRows + 128 * x + row]);
              Lsum += ml.y * (M == -INFINITY ? 0.0f : exp2_approx(ml.x - M));
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float f[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) f[i] = 0.0f;
#pragma unroll 1
              for (int i = 0; i < parts.parts; ++i) {
                const int sl = attn_slot(parts.first + i, i == 0);
                const float w = M == -INFINITY ? 0.0f : exp2_approx(__ldcg(&a.part_ml[sl * kRows + 128 * x + row]).x - M);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 v = __ldcg(part_at(sl, c / 4 + k));
                  f[4 * k] = fmaf(v.x, w, f[4 * k]), f[4 * k + 1] = fmaf(v.y, w, f[4 * k + 1]);
                  f[4 * k + 2] = fmaf(v.z, w, f[4 * k + 2]), f[4 * k + 3] = fmaf(v.w, w, f[4 * k + 3]);
                }
              }
              put(c, f, Lsum > 0.0f ? 1.0f / Lsum : 0.0f);
            }
            put_lse(M, Lsum);
          }
        }
      }
      unit += take;
      u += take;
      if (u < share.end) cur.next(a);
    }
  } else if (warp < 12) {
    // ================================================================ reading the cache
    constexpr int kShares = D / 16;             // lanes of a key: sixteen elements each
    constexpr int kIts = kShares;               // a lane's keys of a unit
    constexpr int kKeysPerIt = 128 / kShares;   // over the four warps
    const int dw = warp - 8;
    const int part = lane % kShares;
    const int r0 = dw * (32 / kShares) + lane / kShares;
    constexpr int kRowBytes = E2M1 ? D / 2 : D;
    constexpr int kBlocks = D / 32;
    Codes<E2M1> kc[kIts], vc[kIts];
    int ks[kIts], vs[kIts];  // scale bytes; -1: nothing there
    // the lane's keys of the unit at key0: cache row of each, or -1
    auto find_rows = [&](int key0, int (&rows)[kIts]) {
      int mine = -1;  // of the 16-key group `lane`
      if (lane < 8) {
        const int key = key0 + 16 * lane;
        if (key < cur.t.hi && key + 16 > cur.t.lo) {
          const int entry = key / a.page_size;
          const int page = __ldg(a.block_table + static_cast<int64_t>(cur.b) * a.max_pages + entry);
          if (page < 0 || page >= a.num_pages) set_status(a.status, MX_ERR_DEVICE_ARG);
          else mine = (page * a.n_kv_heads + cur.head) * a.page_size + (key - entry * a.page_size);
        }
      }
#pragma unroll
      for (int i = 0; i < kIts; ++i) {
        const int r = i * kKeysPerIt + r0;
        const int g = __shfl_sync(0xffffffffu, mine, r / 16);
        const int key = key0 + r;
        rows[i] = g >= 0 && key < cur.t.hi && key >= cur.t.lo ? g + r % 16 : -1;
      }
    };
    auto load = [&](const uint8_t* codes, const uint8_t* scales, const int (&rows)[kIts], Codes<E2M1> (&c)[kIts], int (&s)[kIts]) {
#pragma unroll
      for (int i = 0; i < kIts; ++i) {
        if (rows[i] >= 0) {
          const int64_t r = rows[i];
          c[i].load(codes + r * kRowBytes + part * (kRowBytes / kShares));
          s[i] = __ldg(scales + r * kBlocks + part / 2);
        } else {
          c[i].clear();
          s[i] = -1;
        }
      }
    };
    // sixteen elements as two 16-byte pieces of the swizzled operand; the
    // second panel's lanes write theirs in the other order, so that eight lanes
    // of a store touch all banks
    auto store = [&](uint32_t operand, int i, const uint32_t (&o)[8]) {
      const int r = i * kKeysPerIt + r0;
      uint8_t* line = base + operand + (part / 4) * kPanel + r * 128;
      const int p = (part % 4) * 2;
      const bool swap = part >= 4;
      const uint4 first = make_uint4(o[0], o[1], o[2], o[3]), second = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(line + (((p + (swap ? 1 : 0)) ^ (r & 7)) << 4)) = swap ? second : first;
      *reinterpret_cast<uint4*>(line + (((p + (swap ? 0 : 1)) ^ (r & 7)) << 4)) = swap ? first : second;
    };
    bool ok = true;
    while (ok && u < share.end && cur.b < a.n_seqs) {
      const int take = static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), share.end - u));
      const int first = cur.t.first + cur.place * kUnit;
      int rows[kIts];
      find_rows(first, rows);
      load(a.k_codes, a.k_scales, rows, kc, ks);
      load(a.v_codes, a.v_scales, rows, vc, vs);
      for (int j = 0; j < take && ok; ++j, ++unit) {
        const uint32_t stage = unit & 1u, phase = (unit >> 1) & 1u;
        // the unit's largest scales, and V's smallest of a block that is not zero
        int k_max = -1, v_max = -1, v_min = 255;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          k_max = max(k_max, ks[i]);
          v_max = max(v_max, vs[i]);
          v_min = min(v_min, vs[i] > 0 ? vs[i] : 255);
        }
        k_max = __reduce_max_sync(0xffffffffu, k_max);
        v_max = __reduce_max_sync(0xffffffffu, v_max);
        v_min = __reduce_min_sync(0xffffffffu, v_min);
        int(*seen)[3] = sh.scale_max[stage];
        if (lane == 0) seen[dw][0] = k_max, seen[dw][1] = v_max, seen[dw][2] = v_min;
        named_barrier(3, 128);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          k_max = max(k_max, seen[w][0]);
          v_max = max(v_max, seen[w][1]);
          v_min = min(v_min, seen[w][2]);
        }
        const int k_exp = min(max(k_max - 127, -100), 126), v_exp = min(max(v_max - 127, -100), 126);
        const bool wide = v_exp - (v_min - 127) > 15;
        if (dw == 0 && lane == 0) {
          UnitMeta meta;
          meta.k_scale = __uint_as_float(static_cast<uint32_t>(127 + k_exp) << 23);
          meta.v_exp = v_exp;
          meta.wide = wide;
          sh.meta[unit % kMetaRing] = meta;
        }
        const bool more = j + 1 < take;
        if (more) find_rows(first + (j + 1) * kUnit, rows);

        ok = wait(sh, &sh.k_empty[stage], phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          const uint32_t f = bf16_pow2x2_112(ks[i] - 127 - k_exp);
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] = mul_bf16x2(bf16x2_of_f16x2(kc[i].pair(q)), f);
          store(L::kK + stage * L::kTile, i, o);
        }
        fence_proxy_async_shared();
        mbar_arrive(smem_u32(&sh.k_full[stage]));
        if (more) load(a.k_codes, a.k_scales, rows, kc, ks);

        ok = wait(sh, &sh.v_empty[stage], phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          uint32_t o[8];
          if (wide) {
            const uint32_t f = bf16_pow2x2_112(vs[i] - 127 - v_exp);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = mul_bf16x2(bf16x2_of_f16x2(vc[i].pair(q)), f);
          } else {
            const uint32_t f = f16_pow2x2(vs[i] - 127 - v_exp);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = mul_f16x2(vc[i].pair(q), f);
          }
          store(L::kV + stage * L::kTile, i, o);
        }
        fence_proxy_async_shared();
        mbar_arrive(smem_u32(&sh.v_full[stage]));
        if (more) load(a.v_codes, a.v_scales, rows, vc, vs);
      }
      u += take;
      if (ok && u < share.end) cur.next(a);
    }
  } else {
    // ================================================================ MMAs
    if (lane == 0) {
      const uint32_t q_lo = desc_lo_sw128(smem_u32(base + L::kQ)), k_lo = desc_lo_sw128(smem_u32(base + L::kK));
      // V is MN-major: 64-element panels along N lie kPanel apart (leading
      // offset), eight-key groups 1024 bytes (stride)
      const uint32_t v_lo = ((smem_u32(base + L::kV) >> 4) & 0x3FFFu) | ((kPanel >> 4) << 16);
      const uint32_t qk_idesc = idesc_f16(true, false, 128, kUnit);
      uint32_t q_phase = 0, p_phase = 0;
      bool ok = true;
      auto scores = [&](uint32_t x, uint32_t stage) {
#pragma unroll
        for (uint32_t p = 0; p < D / 64; ++p) {
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            mma_f16_ss(tmem + L::kS + 128u * x, q_lo + ((x * L::kTile + p * kPanel) >> 4) + 2u * k,
                       k_lo + ((stage * L::kTile + p * kPanel) >> 4) + 2u * k, kDescHiSw128, qk_idesc, (p | k) != 0);
        }
        mma_commit(smem_u32(&sh.s_full[x]));
      };
      auto values = [&](uint32_t x, uint32_t stage, uint32_t idesc, bool first) {
#pragma unroll
        for (uint32_t k = 0; k < kUnit / 16; ++k)
          mma_f16_ts(tmem + L::kO + D * x, tmem + L::kS + 128u * x + 8u * k, v_lo + ((stage * L::kTile + k * 2048u) >> 4),
                     kDescHiSw128, idesc, !first || k != 0);
      };
      while (ok && u < share.end && cur.b < a.n_seqs) {
        const int take = static_cast<int>(min(static_cast<int64_t>(cur.t.units - cur.place), share.end - u));
        const bool two = cur.s.n * a.group - cur.tile * kRows > 128;
        ok = wait(sh, &sh.q_full[0], q_phase & 1u, a);
        if (ok && two) ok = wait(sh, &sh.q_full[1], (q_phase >> 1) & 1u, a);
        q_phase ^= two ? 3u : 1u;
        if (ok) ok = wait(sh, &sh.k_full[unit & 1u], (unit >> 1) & 1u, a);
        if (!ok) break;
        tc_fence_after();
        scores(0, unit & 1u);
        if (two) scores(1, unit & 1u);
        mma_commit(smem_u32(&sh.k_empty[unit & 1u]));
        for (int j = 0; j < take; ++j, ++unit) {
          const uint32_t stage = unit & 1u, next = stage ^ 1u;
          const bool more = j + 1 < take;
          ok = wait(sh, &sh.v_full[stage], (unit >> 1) & 1u, a);
          if (ok) ok = wait(sh, &sh.p_full[0], p_phase & 1u, a);
          if (!ok) break;
          tc_fence_after();
          const uint32_t idesc = idesc_f16(sh.meta[unit % kMetaRing].wide != 0, true, 128, D);
          values(0, stage, idesc, j == 0);
          if (more) {
            // P lies in S: this MMA is issued behind the ones that read it
            ok = wait(sh, &sh.k_full[next], ((unit + 1) >> 1) & 1u, a);
            if (!ok) break;
            tc_fence_after();
            scores(0, next);
          } else {
            mma_commit(smem_u32(&sh.o_full[0]));
          }
          if (two) {
            ok = wait(sh, &sh.p_full[1], (p_phase >> 1) & 1u, a);
            if (!ok) break;
            tc_fence_after();
            values(1, stage, idesc, j == 0);
          }
          p_phase ^= two ? 3u : 1u;
          mma_commit(smem_u32(&sh.v_empty[stage]));
          if (more) {
            if (two) scores(1, next);
            mma_commit(smem_u32(&sh.k_empty[next]));
          } else if (two) {
            mma_commit(smem_u32(&sh.o_full[1]));
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, kTmemColumns);
}

template <int D, bool E2M1>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  constexpr int kSmem = Layout<D>::kBytes + 1024;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(k_attn_chunk<D, E2M1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  k_attn_chunk<D, E2M1><<<sms < kMaxCtas ? sms : kMaxCtas, kThreads, kSmem, s>>>(a);
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
