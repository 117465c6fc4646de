// Attention of few new tokens over the paged MX cache (decoding, verifying
// drafts): flash-decoding on register-level MMAs, bound by reading the cache.
//
// A tile is 16 rows (new tokens x the query heads of one KV head), so the
// cache is read once for all heads that share it.  Four warps take 16 keys
// each of a 64-key unit and keep their own running maximum, sum and
// accumulator; they are joined when the CTA's stretch of a segment ends.  Keys
// and values go from global memory to registers and MMA fragments with no
// shared memory between: the contraction order of an MMA is free, so a lane
// feeds it the 16-byte pieces that it loaded.
//
// Arithmetic.  Codes are exact in f16.  A key's blocks are scaled relative to
// the key's largest block scale (a power of two: exact down to 2^-24 of the
// block, 2^-33 of the key's largest element) and that scale multiplies the
// score in fp32; queries are scaled per row to f16's range the same way.  For
// the values the key's largest block scale e joins the exponent of the softmax:
// weights are w = 2^(x + e - M) with M the running maximum of x + e, so that
// both w and the scaled values stay inside f16 whatever the tokens' sizes, and
// the sum is l = sum w 2^-e.  Scores, M, l and the accumulator are fp32; w is
// rounded to f16 (2^-11) for the second MMA.  M moves only when it would grow
// by more than 2^8, which f16 holds: the accumulator is then seldom rescaled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "attn.cuh"
#include "kv.cuh"

namespace mxk {

namespace {

constexpr int kRows = 16;
constexpr int kUnit = 64;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 3;
constexpr int kMinUnits = 4;
constexpr int kCost = 0;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^d as the bits of an f16, d <= 15: subnormal below -14, 0 below -24.
__device__ __forceinline__ uint32_t f16_pow2(int d) {
  return d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : 0x400u >> min(-14 - d, 31);
}

// The largest byte of a row's scale word (kBlocks bytes).
template <int kBlocks>
__device__ __forceinline__ int max_scale(uint32_t w) {
  int m = max(static_cast<int>(w & 0xFFu), static_cast<int>((w >> 8) & 0xFFu));
  if (kBlocks == 4) m = max(m, max(static_cast<int>((w >> 16) & 0xFFu), static_cast<int>(w >> 24)));
  return m;
}

template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[kWords]) {
  if constexpr (kWords == 1) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (kWords == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// One row's scale bytes as a word.
template <int kBlocks>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (kBlocks == 4) return __ldg(reinterpret_cast<const uint32_t*>(p));
  else return __ldg(reinterpret_cast<const uint16_t*>(p));
}

template <int D, bool E2M1>
struct RowsShape {
  static constexpr int kBlocks = D / 32;                    // scales of a row
  static constexpr int kRowBytes = E2M1 ? D / 2 : D;
  static constexpr int kSteps = D / 16;                     // K = 16 steps of a score
  static constexpr int kTiles = D / 8;                      // n = 8 tiles of the output
  static constexpr int kPieces = E2M1 || D == 64 ? 1 : 2;   // loads of a lane's share of a key
  static constexpr int kPieceWords = E2M1 && D == 64 ? 2 : 4;
  static constexpr int kVWords = (E2M1 ? D / 16 : D / 8) / 4;
};

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_attn_rows(const AttnArgs a) {
  using Sh = RowsShape<D, E2M1>;
  __shared__ __align__(16) float s_o[kWarps][kRows][D];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int64_t s_units[kAttnScan];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const AttnShare share = attn_share<kRows, kUnit, kCost, kThreads, false>(a, s_units);
  const int n_heads = a.n_kv_heads * a.group;
  AttnCursor<kRows, kUnit, kCost> cur;
  cur.template start<false>(a, share);

  while (cur.settle(a)) {
    const AttnSeq& s = cur.s;
    const AttnTile& t = cur.t;
    const int head = cur.head, tile = cur.tile, place = cur.place;
    const int take = cur.take();
    const int rows = s.n * a.group;
    const int base = s.kv - s.n;

    // ---------------------------------------------------------------- queries
    // rows g and g + 8; element e of a lane's share is d(e), sixteen at a time
    uint32_t qa[Sh::kSteps][4];
    float row_fac[2];
    int row_lo[2], row_hi[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int R = tile * kRows + g + 8 * r;
      const bool valid = R < rows;
      const int tok = valid ? R / a.group : 0;
      const int hq = head * a.group + (valid ? R - tok * a.group : 0);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(s.q0 + tok) * a.q_stride +
                               static_cast<int64_t>(hq) * D;
      uint32_t w[D / 8];  // the lane's D / 4 elements
#pragma unroll
      for (int p = 0; p < D / 64; ++p) {
        const int d = E2M1 ? c * (D / 4) + 16 * p : c * 16 + 64 * p;
        const uint4* src = reinterpret_cast<const uint4*>(q + d);
        const uint4 x = valid ? __ldg(src) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 y = valid ? __ldg(src + 1) : make_uint4(0u, 0u, 0u, 0u);
        w[8 * p] = x.x, w[8 * p + 1] = x.y, w[8 * p + 2] = x.z, w[8 * p + 3] = x.w;
        w[8 * p + 4] = y.x, w[8 * p + 5] = y.y, w[8 * p + 6] = y.z, w[8 * p + 7] = y.w;
      }
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = max(static_cast<int>(amax >> 7) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);  // 14 - e <= 114
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t h = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
        qa[i / 2][(i & 1) * 2 + r] = h;
      }
      row_fac[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(max(127 + e - 14, 1)) << 23);
      const int at = base + tok;
      row_hi[r] = !valid ? 0 : a.causal ? min(s.kv, at + 1) : s.kv;
      row_lo[r] = a.window > 0 ? max(at - a.window + 1, 0) : 0;
    }
    // keys that every row of the tile sees need no mask
    int all_hi = min(row_hi[0], row_hi[1]), all_lo = max(row_lo[0], row_lo[1]);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, d));
      all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, d));
    }

    // ---------------------------------------------------------------- keys and values
    float o[Sh::kTiles][4];
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    const int32_t* table = a.block_table + static_cast<int64_t>(cur.b) * a.max_pages;
    // Row index of 16 keys from `key` (a page holds a multiple of 16): or -1
    // where there is nothing to read.
    auto find_row = [&](int key) -> int64_t {
      if (key >= t.hi || key + 16 <= t.lo) return -1;
      const int entry = key / a.page_size;
      const int page = __ldg(table + entry);
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
        return -1;
      }
      return (static_cast<int64_t>(page) * a.n_kv_heads + head) * a.page_size + (key - entry * a.page_size);
    };
    uint32_t kw[2][Sh::kPieces][Sh::kPieceWords], ks[2], vw[4][Sh::kVWords], vs[4];
    auto load_k = [&](int64_t row) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t r = row + 8 * j + g;
#pragma unroll
        for (int p = 0; p < Sh::kPieces; ++p)
          load_words(a.k_codes + r * Sh::kRowBytes + c * (4 * Sh::kPieceWords) + 64 * p, kw[j][p]);
        ks[j] = load_scales<Sh::kBlocks>(a.k_scales + r * Sh::kBlocks);
      }
    };
    // the keys of the lane's score columns: 2c, 2c + 1, 8 + 2c, 9 + 2c
    auto load_v = [&](int64_t row) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = row + 8 * (j >> 1) + 2 * c + (j & 1);
        load_words(a.v_codes + r * Sh::kRowBytes + g * (4 * Sh::kVWords), vw[j]);
        vs[j] = load_scales<Sh::kBlocks>(a.v_scales + r * Sh::kBlocks);
      }
    };

    int key = t.first + place * kUnit + warp * 16;
    const int key_end = t.first + (place + take) * kUnit;
    int64_t row = key < key_end ? find_row(key) : -1;
    if (row >= 0) {
      load_k(row);
      load_v(row);
    }
    for (; key < key_end; key += kUnit) {
      const int64_t next = key + kUnit < key_end ? find_row(key + kUnit) : -1;
      if (row < 0) {
        row = next;
        if (row >= 0) {
          load_k(row);
          load_v(row);
        }
        continue;
      }
      // scores of 2 x 8 keys
      float x[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int top = max_scale<Sh::kBlocks>(ks[j]);
        uint32_t mult[D / 64];  // of the lane's 16-element groups
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
          const int blk = E2M1 ? (D == 128 ? c : c >> 1) : (c >> 1) + 2 * p;
          mult[p] = f16_pow2(static_cast<int>((ks[j] >> (8 * blk)) & 0xFFu) - top) * 0x10001u;
        }
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < Sh::kSteps; ++st) {
          uint32_t b0, b1;
          if (E2M1) {
            const uint32_t w = kw[j][0][st / 2] >> ((st & 1) * 16);
            b0 = f16x2_of_e2m1x2(w & 0xFFu);
            b1 = f16x2_of_e2m1x2((w >> 8) & 0xFFu);
          } else {
            const uint32_t w = kw[j][st / 4][st % 4];
            b0 = f16x2_of_e4m3x2(w & 0xFFFFu);
            b1 = f16x2_of_e4m3x2(w >> 16);
          }
          mma_f16(acc, qa[st], mul2(b0, mult[st / 4]), mul2(b1, mult[st / 4]));
        }
        const float key_fac = e8m0_value(top);
        const float f0 = __shfl_sync(0xffffffffu, key_fac, 8 * c), f1 = __shfl_sync(0xffffffffu, key_fac, 8 * c + 4);
        x[j][0] = acc[0] * (row_fac[0] * f0);
        x[j][1] = acc[1] * (row_fac[0] * f1);
        x[j][2] = acc[2] * (row_fac[1] * f0);
        x[j][3] = acc[3] * (row_fac[1] * f1);
      }
      if (next >= 0) load_k(next);
      // exponents of the values' keys; masks
      float e_inv[4];
      uint32_t v_mult[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = min(max(max_scale<Sh::kBlocks>(vs[j]) - 127, -100), 126);
        const int blk = D == 128 ? g >> 1 : g >> 2;
        v_mult[j] = f16_pow2(min(static_cast<int>((vs[j] >> (8 * blk)) & 0xFFu) - 127 - e, 2));
        e_inv[j] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float ef = static_cast<float>(e);
        x[j >> 1][j & 1] += ef;
        x[j >> 1][2 + (j & 1)] += ef;
      }
      if (key + 16 > all_hi || key < all_lo) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = key + 8 * (j >> 1) + 2 * c + (j & 1);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (at >= row_hi[r] || at < row_lo[r]) x[j >> 1][2 * r + (j & 1)] = -INFINITY;
          // a place that no row sees may hold anything, NaN included
          if (at >= t.hi || at < t.lo) {
#pragma unroll
            for (int i = 0; i < Sh::kVWords; ++i) vw[j][i] = 0u;
          }
        }
      }
      // running maximum
      float top[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.0f || top[1] > m[1] + 8.0f)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float to = fmaxf(m[r], top[r]);
          const float f = to == -INFINITY ? 1.0f : exp2_approx(m[r] - to);
          m[r] = to;
          l[r] *= f;
#pragma unroll
          for (int i = 0; i < Sh::kTiles; ++i) {
            o[i][2 * r] *= f;
            o[i][2 * r + 1] *= f;
          }
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float from = m[r] == -INFINITY ? 0.0f : m[r];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = exp2_approx(x[j >> 1][2 * r + (j & 1)] - from);
          l[r] = fmaf(w[j], e_inv[j], l[r]);
        }
        pa[r] = pack_f16(w[0], w[1]);
        pa[2 + r] = pack_f16(w[2], w[3]);
      }
      const uint32_t m01 = v_mult[0] | (v_mult[1] << 16), m23 = v_mult[2] | (v_mult[3] << 16);
#pragma unroll
      for (int i = 0; i < Sh::kVWords; ++i) {
        if (E2M1) {
          // low nibbles are the even elements; a byte pairs one element of two keys
          const uint32_t even01 = (vw[0][i] & 0x0F0F0F0Fu) | ((vw[1][i] & 0x0F0F0F0Fu) << 4);
          const uint32_t odd01 = ((vw[0][i] >> 4) & 0x0F0F0F0Fu) | (vw[1][i] & 0xF0F0F0F0u);
          const uint32_t even23 = (vw[2][i] & 0x0F0F0F0Fu) | ((vw[3][i] & 0x0F0F0F0Fu) << 4);
          const uint32_t odd23 = ((vw[2][i] >> 4) & 0x0F0F0F0Fu) | (vw[3][i] & 0xF0F0F0F0u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma_f16(o[8 * i + 2 * k], pa, mul2(f16x2_of_e2m1x2((even01 >> (8 * k)) & 0xFFu), m01),
                    mul2(f16x2_of_e2m1x2((even23 >> (8 * k)) & 0xFFu), m23));
            mma_f16(o[8 * i + 2 * k + 1], pa, mul2(f16x2_of_e2m1x2((odd01 >> (8 * k)) & 0xFFu), m01),
                    mul2(f16x2_of_e2m1x2((odd23 >> (8 * k)) & 0xFFu), m23));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t sel = k == 0 ? 0x5140u : 0x7362u;
            const uint32_t y01 = __byte_perm(vw[0][i], vw[1][i], sel), y23 = __byte_perm(vw[2][i], vw[3][i], sel);
            mma_f16(o[4 * i + 2 * k], pa, mul2(f16x2_of_e4m3x2(y01 & 0xFFFFu), m01),
                    mul2(f16x2_of_e4m3x2(y23 & 0xFFFFu), m23));
            mma_f16(o[4 * i + 2 * k + 1], pa, mul2(f16x2_of_e4m3x2(y01 >> 16), m01),
                    mul2(f16x2_of_e4m3x2(y23 >> 16), m23));
          }
        }
      }
      if (next >= 0) load_v(next);
      row = next;
    }

    // ---------------------------------------------------------------- join the warps
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        s_m[warp][g + 8 * r] = m[r];
        s_l[warp][g + 8 * r] = l[r];
      }
      // column n of output tile i is element n * D / 8 + i
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < Sh::kTiles; i += 4)
          *reinterpret_cast<float4*>(&s_o[warp][g + 8 * r][(2 * c + k) * (D / 8) + i]) =
              make_float4(o[i][2 * r + k], o[i + 1][2 * r + k], o[i + 2][2 * r + k], o[i + 3][2 * r + k]);
      }
    }
    __syncthreads();

    const bool whole = take == t.units;
    const AttnParts p = attn_parts(share, cur.u - place, t.units);
    const int slot = attn_slot(blockIdx.x, place == 0);

    // writes a finished row: four elements a lane
    auto finish = [&](int r, int d4, float4 acc, float M, float L) {
      const int R = tile * kRows + r;
      const int tok = R / a.group;
      const int64_t oh = static_cast<int64_t>(s.q0 + tok) * n_heads + head * a.group + (R - tok * a.group);
      const float inv = L > 0.0f ? 1.0f / L : 0.0f;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&lo);
      w.y = *reinterpret_cast<const uint32_t*>(&hi);
      reinterpret_cast<uint2*>(a.out)[oh * (D / 4) + d4] = w;
      if (a.lse && d4 == 0) a.lse[oh] = L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
    };
    constexpr int kLanes = D / 4;  // lanes of a row
    for (int i = tid; i < kRows * kLanes; i += kThreads) {
      const int r = i / kLanes, d4 = i - r * kLanes;
      if (tile * kRows + r >= rows) continue;
      float M = s_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float L = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = M == -INFINITY ? 0.0f : exp2_approx(s_m[w][r] - M);
        const float4 v = *reinterpret_cast<const float4*>(&s_o[w][r][4 * d4]);
        L = fmaf(s_l[w][r], f, L);
        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        finish(r, d4, acc, M, L);
      } else {
        reinterpret_cast<float4*>(a.part_o)[(static_cast<int64_t>(slot) * kRows + r) * kLanes + d4] = acc;
        if (d4 == 0) a.part_ml[slot * kRows + r] = make_float2(M, L);
      }
    }
    if (!whole) {
      // ---------------------------------------------------------------- join the CTAs
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(&a.arrived[p.first], 1u) == static_cast<unsigned>(p.parts - 1);
      __syncthreads();
      if (s_last) {
        __threadfence();
        auto slot_of = [&](int i) { return attn_slot(p.first + i, i == 0); };
        for (int r = warp; r < kRows && tile * kRows + r < rows; r += kWarps) {
          float M = -INFINITY;
          for (int i = lane; i < p.parts; i += 32) M = fmaxf(M, __ldcg(&a.part_ml[slot_of(i) * kRows + r]).x);
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          float L = 0.0f;
          float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int i = 0; i < p.parts; ++i) {
            const int sl = slot_of(i);
            const float2 ml = __ldcg(&a.part_ml[sl * kRows + r]);
            const float f = M == -INFINITY ? 0.0f : exp2_approx(ml.x - M);
            L = fmaf(ml.y, f, L);
            if (lane < kLanes) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (static_cast<int64_t>(sl) * kRows + r) * kLanes + lane);
              acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
              acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
            }
          }
          if (lane < kLanes) finish(r, lane, acc, M, L);
        }
        if (tid == 0) a.arrived[p.first] = 0u;  // ready for the next launch
      }
    }
    __syncthreads();  // the warps' parts are read before the next segment overwrites them
    cur.pass(take);
  }
}

template <int D, bool E2M1>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = attn_sm_count(&sms);
  if (e != cudaSuccess) return e;
  k_attn_rows<D, E2M1><<<sms * kCtasPerSm < kAttnMaxCtas ? sms * kCtasPerSm : kAttnMaxCtas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

size_t attn_rows_part_bytes(int head_dim) {
  return static_cast<size_t>(2) * kAttnMaxCtas * kRows * (sizeof(float2) + sizeof(float) * head_dim);
}

cudaError_t launch_attn_rows(AttnArgs a, cudaStream_t s) {
  a.min_units = kMinUnits;
  a.part_o = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2) * kAttnMaxCtas * kRows);
  if (a.head_dim == 128) return a.e2m1 ? launch<128, true>(a, s) : launch<128, false>(a, s);
  return a.e2m1 ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace mxk
