// Attention of few new tokens over the paged MX cache (decoding, verifying
// drafts): the keys split over all SMs, one pass with a running softmax, on
// register-level MMAs (with the rows as M a tensor-memory tile of 128 would be 94%
// empty; one with the keys as M was not built).
//
// A tile is 8 rows (new tokens x the query heads of one KV head), so the
// cache is read once for all heads that share it.  A fifth warp fetches units of
// 64 keys ahead by TMA, over the segments' borders; four warps take 16 keys each
// of a unit and keep their own running maximum, sum and accumulator, joined when
// the CTA's stretch of a segment ends.
//
// What bounds it.  With MXFP8 the cache's bytes: of what 64 instead of 32
// sequences of 8192 add, 6.6 TB/s (98% of a copy's).  A call has 17 us beside
// that: 4 until every CTA knows its stretch, 2 until the first keys are there, 4
// to join, launch and uneven ends; so 32 ragged sequences of up to 8192 (300 MB)
// take 62 us where a copy of the bytes takes 44, and 6 drafts over 2051 keys 17.
// With MXFP4 the instructions: half the bytes a key and 514 instructions for 16
// keys of a warp (a whole call's, by the counter), with the pipe of conversions and
// bit operations busy for 63% of the cycles: 3.2 TB/s; 3 sequences of up to 65536
// take 79 us (copy: 32).
//
// Both products are transposed, S^T = K Q^T and O^T += V^T P^T, so that the query
// rows are the MMAs' columns, of which there are 8 where there are 16 rows of
// keys or elements.  More rows are more tiles, which read the keys again, mostly
// from L2: tiles of 16 rows share the widened codes, but their registers spill
// (8 sequences of 8192 and 4 KV heads, 16 rows: 53 us, as two tiles 35).  P^T goes
// from the layout of S^T's results to that of an operand by a transposing move.
// The contraction order of an MMA is free, so a lane feeds it the 16-byte pieces
// that it reads from shared memory.  (Register-level MMAs on the 8-bit codes were
// slower than widening them for f16 ones: 32 sequences took 84 us against 77.)
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
#include <atomic>
#include <climits>
#include <cstdint>

#include "attn.cuh"
#include "kv.cuh"

namespace mxk {

namespace {

constexpr int kRows = 8;                   // of a tile
constexpr int kUnit = 64;
constexpr int kWarps = 4;                  // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kCtasPerSm = 3;              // what the registers allow: 160 threads of 128
// Places of a CTA's stretch at least (6 drafts over 2051 keys: 17.0 us with 4, 16.7
// with 2, 16.8 with 6).
constexpr int kMinUnits = 4;
// A segment's queries and output, in units (32 sequences of up to 8192: 72 us with
// 1, 63 with 4, 62 with 8, 66 with 16).
constexpr int kCost = 8;

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

// A word's four even or odd E2M1 codes as E4M3 codes of 2^-6 their size, by moving
// their bits; the conversion to f16 then starts from E4M3 (3 sequences of up to
// 65536: 83 us converting from E2M1 itself, 82 moving its bits into f16, 79 this way).
constexpr int kE2m1Shift = 6;
__device__ __forceinline__ uint32_t e4m3_of_even(uint32_t w) { return (w << 4 & 0x80808080u) | (w << 2 & 0x1C1C1C1Cu); }
__device__ __forceinline__ uint32_t e4m3_of_odd(uint32_t w) { return (w & 0x80808080u) | (w >> 2 & 0x1C1C1C1Cu); }

// The warp's 8 x 8 matrix of 16-bit elements, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The float 2^d, 0 below -126.
__device__ __forceinline__ float pow2_or_zero(int d) { return __uint_as_float(static_cast<uint32_t>(max(127 + d, 0)) << 23); }

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
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// One row's scale bytes as a word.
template <int kBlocks>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p, int row) {
  if constexpr (kBlocks == 4) return reinterpret_cast<const uint32_t*>(p)[row];
  else return reinterpret_cast<const uint16_t*>(p)[row];
}

template <int D, bool E2M1>
struct RowsShape {
  static constexpr int kBlocks = D / 32;                    // scales of a row
  static constexpr int kRowBytes = E2M1 ? D / 2 : D;
  static constexpr int kTiles = D / 16;                     // m = 16 tiles of the output
  static constexpr int kSteps = D / 16;                     // K = 16 steps of a score
  // a lane's D / 4 elements of a key of K, from c * D / 4 on, and its D / 8 of a
  // key of V, from g * D / 8 on
  static constexpr int kPieces = E2M1 || D == 64 ? 1 : 2;
  static constexpr int kPieceWords = E2M1 && D == 64 ? 2 : 4;
  static constexpr int kVWords = kRowBytes / 32;
  // a stage: K's codes, V's, K's scales, V's
  static constexpr uint32_t kCodes = kUnit * kRowBytes, kScales = kUnit * kBlocks;
  static constexpr uint32_t kStage = (2 * kCodes + 2 * kScales + 1023) / 1024 * 1024;
  static constexpr int kStages = 53248 / kStage < 6 ? 53248 / kStage : 6;  // three CTAs share an SM
  static constexpr uint32_t kJoin = 2 * kRows * D * sizeof(float);
  static constexpr uint32_t kBytes = kStages * kStage + kJoin;
  // where byte `b` of row r lies in a stage, as the TMA's swizzle puts it
  static __device__ __forceinline__ uint32_t at(int r, int b) {
    const int piece = b / 16;
    const int moved = kRowBytes == 128 ? piece ^ (r & 7) : kRowBytes == 64 ? piece ^ ((r >> 1) & 3) : piece ^ ((r >> 2) & 1);
    return static_cast<uint32_t>(r * kRowBytes + moved * 16 + b % 16);
  }
};

// AttnCursor::settle, out of line: once a segment.
template <class Cursor>
__device__ __noinline__ bool settle(Cursor& c, const AttnArgs& a) {
  return c.settle(a);
}
// The compute warps meet.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// What the scales of a warp's 16 keys say, worked out half a key a lane.
struct KeyTable {
  float4 key[16];          // K's largest scale; V's largest scale's exponent e, 2^-e
  uint32_t k_rel[4][16];   // a block's K scale relative to the key's largest, in f16, twice
  __half v_rel[4][16];     // a block's V scale relative to the key's largest
};

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    k_attn_rows(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
  using Sh = RowsShape<D, E2M1>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[Sh::kStages], empty[Sh::kStages];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ uint2 s_q[Sh::kSteps][32];
  __shared__ __align__(16) KeyTable s_table[kWarps];
  __shared__ int s_e[kRows];
  __shared__ uint32_t s_here[Sh::kStages];  // 16-key groups that are there
  __shared__ uint32_t s_units[kAttnScan];
  __shared__ volatile int failed;
  __shared__ int s_last;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* s_o = reinterpret_cast<float*>(base + Sh::kStages * Sh::kStage);  // [2][kRows][D]
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kWarps);
    }
    failed = 0;
    fence_mbar_init();
  }
  const AttnShare share = attn_share<kRows, kUnit, kCost, kThreads, false>(a, s_units);  // its barriers cover the above
  const int n_heads = a.n_kv_heads * a.group;
  AttnCursor<kRows, kUnit, kCost, 1> cur;
  cur.template start<false>(a, share);
  Ring<Sh::kStages> ring;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- fetching
    constexpr int kGroups = kUnit / 16;
    const int group = lane % kGroups, kind = lane / kGroups;  // K's codes, V's, K's scales, V's
    const bool leads = 16 * group % a.box_keys == 0;
    const int none = a.num_pages * a.n_kv_heads * a.page_size;
    if (lane < 2) prefetch_tensormap(lane == 0 ? &k_map : &v_map);
    AttnWalk<kUnit> walk;
    int issued = 0;
    bool ok = true;
    while (ok && settle(cur, a)) {
      const int take = cur.take();
      walk.start(a, cur, group);
#pragma unroll 1
      for (int i = 0; i < take; ++i) {
        uint32_t here, bad;
        const int row = walk.box(a, cur.head, group, here, bad);
        const uint32_t boxes = __ballot_sync(0xffffffffu, leads && row >= 0) & ((1u << kGroups) - 1);
        ok = attn_wait<true>(&failed, &empty[ring.stage], ring.phase ^ 1u, a);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = smem_u32(&full[ring.stage]);
        if (lane == 0) {
          s_here[ring.stage] = here;
          mbar_arrive_expect_tx(bar, 2 * Sh::kCodes + 2 * __popc(boxes) * (a.box_keys * Sh::kBlocks));
        }
        __syncwarp();
        const uint32_t to = smem_u32(base + ring.stage * Sh::kStage);
        if (leads && kind < 2) {
          // a box that is not there is read past the table's end: zeros
          tma_load_2d(to + kind * Sh::kCodes + group * (Sh::kCodes / kGroups), kind == 0 ? &k_map : &v_map, 0,
                      row < 0 ? none : row, bar);
        } else if (leads && kind < 4 && row >= 0) {
          bulk_load(to + 2 * Sh::kCodes + (kind - 2) * Sh::kScales + group * (Sh::kScales / kGroups),
                    (kind == 2 ? a.k_scales : a.v_scales) + static_cast<int64_t>(row) * Sh::kBlocks, a.box_keys * Sh::kBlocks, bar);
        }
        __syncwarp();
        ++issued;
        ring.next();
        walk.step(a);
      }
      cur.pass(take);
    }
    // the last fills have landed before the CTA exits, also where a wait of the
    // others ran out
    for (int i = issued > Sh::kStages ? issued - Sh::kStages : 0; i < issued; ++i)
      mbar_wait(smem_u32(&full[i % Sh::kStages]), (i / Sh::kStages) & 1u, 100000000ull);
    return;
  }

  KeyTable& table = s_table[warp];
  const int half = lane >> 4;  // of the blocks of key lane % 16, whose scales the lane works out
  // where the lane's codes lie in a stage
  int k_off[Sh::kPieces], v_off[2];
#pragma unroll
  for (int p = 0; p < Sh::kPieces; ++p) k_off[p] = Sh::at(warp * 16 + g, c * (Sh::kRowBytes / 4) + 16 * p);
#pragma unroll
  for (int p = 0; p < 2; ++p) v_off[p] = Sh::at(warp * 16 + 2 * c + p, g * (Sh::kRowBytes / 8));

  bool ok = true;
  while (settle(cur, a)) {
    const AttnSeq s = cur.s;
    const AttnTile t = cur.t;
    const int head = cur.head, tile = cur.tile, place = cur.place;
    const int take = cur.take();
    const int rows = s.n * a.group;
    const int old = s.kv - s.n;  // the position of the first new token

    // ---------------------------------------------------------------- queries
    // as the scores' B fragments, a row's largest element scaled to [2^14, 2^15)
    if (warp == 0) {
      const int R = tile * kRows + g;
      const bool valid = R < rows;
      const int tok = valid ? a.group_div.of(R) : 0;
      const int hq = head * a.group + (valid ? R - tok * a.group : 0);
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                      static_cast<int64_t>(s.q0 + tok) * a.q_stride +
                                                      static_cast<int64_t>(hq) * D + c * (D / 4));
      uint4 w[D / 32];  // the lane's D / 4 elements
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = valid ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) amax = max(amax, max(e[k] & 0x7FFFu, (e[k] >> 16) & 0x7FFFu));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = max(static_cast<int>(amax >> 7) - 127, -100);
      // 14 - e <= 114; a row with an infinity or NaN has no scores
      const float up = e == 128 ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[2 * k] = __uint_as_float(x[k] << 16) * up;
          f[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u) * up;
        }
        uint32_t y[4];  // E2M1: the even elements, then the odd ones, as they come from a word of K
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = E2M1 ? pack_f16(f[4 * (k & 1) + k / 2], f[4 * (k & 1) + 2 + k / 2]) : pack_f16(f[2 * k], f[2 * k + 1]);
        s_q[2 * i][lane] = make_uint2(y[0], y[1]);
        s_q[2 * i + 1][lane] = make_uint2(y[2], y[3]);
      }
      if (c == 0) s_e[g] = e;
    }
    meet();
    // of the lane's rows 2 c + k
    float row_fac[2];
    int row_lo[2], row_hi[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int R = tile * kRows + 2 * c + k;
      const int at = old + a.group_div.of(R);
      row_fac[k] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(max(127 + s_e[2 * c + k] - 14, 1)) << 23);
      // rows past the tile's are zeros that nobody reads
      row_hi[k] = R >= rows ? INT_MAX : a.causal ? min(s.kv, at + 1) : s.kv;
      row_lo[k] = R < rows && a.window > 0 ? attn_row_lo(a, at) : 0;
    }
    // keys in [all_lo, all_hi) need no mask
    const int all_hi = __reduce_min_sync(0xffffffffu, min(row_hi[0], row_hi[1]));
    const int all_lo = __reduce_max_sync(0xffffffffu, max(row_lo[0], row_lo[1]));
    uint2 qb[Sh::kSteps];
#pragma unroll
    for (int st = 0; st < Sh::kSteps; ++st) qb[st] = s_q[st][lane];

    // ---------------------------------------------------------------- keys and values
    // o[i][k + 2 d]: row 2 c + k, element g * D / 8 + 2 i + d
    float o[Sh::kTiles][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

#pragma unroll 1
    for (int i = 0; i < take; ++i, ring.next()) {
      const int key = t.first + (place + i) * kUnit + warp * 16;
      if (ok) ok = attn_wait<true>(&failed, &full[ring.stage], ring.phase, a);
      ok = __all_sync(0xffffffffu, ok);
      // Behind a wait that ran out a warp releases nothing: stages that it never saw
      // full would be filled again over copies in flight, and their barriers get an
      // arrival too many.  The fetching warp's next wait then gives up too.
      if (!ok) continue;
      if (!(s_here[ring.stage] >> warp & 1u)) {
        warp_arrive(&empty[ring.stage]);
        continue;
      }
      const uint8_t* k_codes = base + ring.stage * Sh::kStage;
      const uint8_t* v_codes = k_codes + Sh::kCodes;
      const uint8_t* k_scales = v_codes + Sh::kCodes;
      const uint8_t* v_scales = k_scales + Sh::kScales;
      uint32_t kw[2][Sh::kPieces][Sh::kPieceWords], vw[4][Sh::kVWords];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < Sh::kPieces; ++p) load_words(k_codes + k_off[p] + j * 8 * Sh::kRowBytes, kw[j][p]);
      // the keys 2c, 2c + 1, 8 + 2c, 9 + 2c of the lane's operands
#pragma unroll
      for (int j = 0; j < 4; ++j) load_words(v_codes + v_off[j & 1] + (j >> 1) * 8 * Sh::kRowBytes, vw[j]);
      {
        const uint32_t ks = load_scales<Sh::kBlocks>(k_scales, warp * 16 + (lane & 15));
        const uint32_t vs = load_scales<Sh::kBlocks>(v_scales, warp * 16 + (lane & 15));
        const int k_top = max_scale<Sh::kBlocks>(ks), v_top = max_scale<Sh::kBlocks>(vs), e = min(max(v_top - 127, -100), 126);
        constexpr int kHalf = Sh::kBlocks / 2, kShift = E2M1 ? kE2m1Shift : 0;
        const uint32_t kh = ks >> (8 * kHalf * half), vh = vs >> (8 * kHalf * half);
#pragma unroll
        for (int b = 0; b < kHalf; ++b) {
          const float kr = pow2_or_zero(static_cast<int>((kh >> (8 * b)) & 0xFFu) - k_top + kShift);
          table.k_rel[kHalf * half + b][lane & 15] = pack_f16(kr, kr);
          table.v_rel[kHalf * half + b][lane & 15] =
              __float2half_rn(pow2_or_zero(min(static_cast<int>((vh >> (8 * b)) & 0xFFu) - 127 - e, 1) + kShift));
        }
        // a scale that is NaN: K's makes the score NaN, V's the row's sum
        table.key[lane & 15] = make_float4(e8m0_value(k_top), static_cast<float>(e),
                                           __uint_as_float(v_top == 255 ? 0x7FC00000u : static_cast<uint32_t>(127 - e) << 23), 0.0f);
        __syncwarp();
      }
      // scores of keys g and g + 8 for the lane's rows
      const int k_blk = D == 128 ? c : c >> 1;  // of the lane's elements
      const uint32_t k_mult[2] = {table.k_rel[k_blk][g], table.k_rel[k_blk][g + 8]};
      float x[4] = {};
#pragma unroll
      for (int st = 0; st < Sh::kSteps; ++st) {
        uint32_t ka[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t b0, b1;
          // E2M1: a word of eight elements for two steps, the even ones first; the
          // queries lie in the same order
          uint32_t w;
          if (E2M1) w = st & 1 ? e4m3_of_odd(kw[j][0][st / 2]) : e4m3_of_even(kw[j][0][st / 2]);
          else w = kw[j][st / 4][st % 4];
          b0 = f16x2_of_e4m3x2(w & 0xFFFFu);
          b1 = f16x2_of_e4m3x2(w >> 16);
          ka[j] = mul2(b0, k_mult[j]);
          ka[2 + j] = mul2(b1, k_mult[j]);
        }
        mma_f16(x, ka, qb[st].x, qb[st].y);
      }
      float4 key4[2] = {table.key[g], table.key[g + 8]};
      // x[2 j + k]: key g + 8 j, row 2 c + k
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(x[i], row_fac[i & 1] * key4[i >> 1].x, key4[i >> 1].y);
      if (key + 16 > all_hi || key < all_lo) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = key + g + 8 * (i >> 1);
          if (at >= row_hi[i & 1] || at < row_lo[i & 1]) x[i] = -INFINITY;
        }
        // a place that no row sees may hold anything, NaN included
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = key + 8 * (j >> 1) + 2 * c + (j & 1);
          if (at >= t.hi || at < t.lo) {
#pragma unroll
            for (int i = 0; i < Sh::kVWords; ++i) vw[j][i] = 0u;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (key + g + 8 * j >= t.hi || key + g + 8 * j < t.lo) key4[j].z = 0.0f;
      }
      // running maximum
      const bool above = fmaxf(x[0], x[2]) > m[0] + 8.0f || fmaxf(x[1], x[3]) > m[1] + 8.0f;
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float to = fmaxf(x[k], x[2 + k]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
          to = fmaxf(to, m[k]);
          const float f = to == -INFINITY ? 1.0f : exp2_approx(m[k] - to);
          m[k] = to;
          l[k] *= f;
#pragma unroll
          for (int i = 0; i < Sh::kTiles; ++i) {
            o[i][k] *= f;
            o[i][2 + k] *= f;
          }
        }
      }
      const float from[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
      uint32_t pb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[k] = exp2_approx(x[2 * j + k] - from[k]);
          l[k] = fmaf(w[k], key4[j].z, l[k]);
        }
        pb[j] = transposed(pack_f16(w[0], w[1]));
      }
      const int v_blk = D == 128 ? g >> 1 : g >> 2;
      const uint32_t rel[2] = {*reinterpret_cast<const uint32_t*>(&table.v_rel[v_blk][2 * c]),
                               *reinterpret_cast<const uint32_t*>(&table.v_rel[v_blk][8 + 2 * c])};
      // two elements (rows g and g + 8 of the MMA) of keys 0, 1 and 2, 3
      auto values = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        const uint32_t va[4] = {mul2(a0, rel[0]), mul2(a1, rel[0]), mul2(a2, rel[1]), mul2(a3, rel[1])};
        mma_f16(o[i], va, pb[0], pb[1]);
      };
#pragma unroll
      for (int i = 0; i < Sh::kVWords; ++i) {
        // an element of two keys side by side, two such in a word
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t sel = k == 0 ? 0x5140u : 0x7362u;
          if (E2M1) {
            const uint32_t even01 = __byte_perm(e4m3_of_even(vw[0][i]), e4m3_of_even(vw[1][i]), sel);
            const uint32_t even23 = __byte_perm(e4m3_of_even(vw[2][i]), e4m3_of_even(vw[3][i]), sel);
            const uint32_t odd01 = __byte_perm(e4m3_of_odd(vw[0][i]), e4m3_of_odd(vw[1][i]), sel);
            const uint32_t odd23 = __byte_perm(e4m3_of_odd(vw[2][i]), e4m3_of_odd(vw[3][i]), sel);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              values(4 * i + 2 * k + h, f16x2_of_e4m3x2(even01 >> (16 * h) & 0xFFFFu), f16x2_of_e4m3x2(odd01 >> (16 * h) & 0xFFFFu),
                     f16x2_of_e4m3x2(even23 >> (16 * h) & 0xFFFFu), f16x2_of_e4m3x2(odd23 >> (16 * h) & 0xFFFFu));
          } else {
            const uint32_t y01 = __byte_perm(vw[0][i], vw[1][i], sel), y23 = __byte_perm(vw[2][i], vw[3][i], sel);
            values(2 * i + k, f16x2_of_e4m3x2(y01 & 0xFFFFu), f16x2_of_e4m3x2(y01 >> 16), f16x2_of_e4m3x2(y23 & 0xFFFFu),
                   f16x2_of_e4m3x2(y23 >> 16));
          }
        }
      }
      warp_arrive(&empty[ring.stage]);
    }

    // ---------------------------------------------------------------- join the warps
    // in two steps: warps 2 and 3 hand theirs to 0 and 1
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
      if (g == 0) {
        s_m[warp][2 * c + k] = m[k];
        s_l[warp][2 * c + k] = l[k];
      }
    }
    auto mine = [&](int k, int i) {
      return reinterpret_cast<float4*>(s_o + ((warp & 1) * kRows + 2 * c + k) * D + g * (D / 8) + 2 * i);
    };
    if (warp >= 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < Sh::kTiles; i += 2) *mine(k, i) = make_float4(o[i][k], o[i][2 + k], o[i + 1][k], o[i + 1][2 + k]);
    }
    meet();
    if (warp < 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float other = s_m[warp + 2][2 * c + k], M = fmaxf(m[k], other), from = M == -INFINITY ? 0.0f : M;
        const float f = exp2_approx(m[k] - from), h = exp2_approx(other - from);
#pragma unroll
        for (int i = 0; i < Sh::kTiles; i += 2) {
          const float4 v = *mine(k, i);
          *mine(k, i) = make_float4(fmaf(o[i][k], f, v.x * h), fmaf(o[i][2 + k], f, v.y * h), fmaf(o[i + 1][k], f, v.z * h),
                                    fmaf(o[i + 1][2 + k], f, v.w * h));
        }
      }
    }
    meet();

    const bool whole = take == t.units;
    const AttnParts p = attn_parts<1>(share, cur.u - place, t.units);
    const int slot = attn_slot(blockIdx.x, place == 0);

    // writes a finished row: four elements a lane
    auto finish = [&](int r, int d4, float4 acc, float M, float L) {
      const int R = tile * kRows + r;
      const int tok = a.group_div.of(R);
      const int64_t oh = static_cast<int64_t>(s.q0 + tok) * n_heads + head * a.group + (R - tok * a.group);
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&lo);
      w.y = *reinterpret_cast<const uint32_t*>(&hi);
      reinterpret_cast<uint2*>(a.out)[oh * (D / 4) + d4] = w;
      if (a.lse && d4 == 0) a.lse[oh] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    };
    constexpr int kLanes = D / 4;  // lanes of a row
    for (int i = tid; i < kRows * kLanes; i += 32 * kWarps) {
      const int r = i / kLanes, d4 = i - r * kLanes;
      if (tile * kRows + r >= rows) continue;
      const float m0 = fmaxf(s_m[0][r], s_m[2][r]), m1 = fmaxf(s_m[1][r], s_m[3][r]);
      const float M = fmaxf(m0, m1), from = M == -INFINITY ? 0.0f : M;
      float L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L = fmaf(s_l[w][r], exp2_approx(s_m[w][r] - from), L);
      const float f0 = exp2_approx(m0 - from), f1 = exp2_approx(m1 - from);
      const float4 v0 = *reinterpret_cast<const float4*>(s_o + r * D + 4 * d4);
      const float4 v1 = *reinterpret_cast<const float4*>(s_o + (kRows + r) * D + 4 * d4);
      const float4 acc = make_float4(fmaf(v0.x, f0, v1.x * f1), fmaf(v0.y, f0, v1.y * f1), fmaf(v0.z, f0, v1.z * f1),
                                     fmaf(v0.w, f0, v1.w * f1));
      if (whole) {
        finish(r, d4, acc, M, L);
      } else {
        reinterpret_cast<float4*>(a.part_o)[(static_cast<int64_t>(slot) * kRows + r) * kLanes + d4] = acc;
        if (d4 == 0) a.part_ml[slot * kRows + r] = make_float2(M, L);
      }
    }
    if (!whole) {
      // ---------------------------------------------------------------- join the CTAs
      // also after a wait that ran out: the counters are zero for the next call
      meet();
      if (tid == 0) s_last = attn_arrive(&a.arrived[p.first]) == static_cast<unsigned>(p.parts - 1);
      meet();
      if (s_last) {
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
    meet();  // the warps' parts are read before the next segment overwrites them
    cur.pass(take);
  }
}

template <int D, bool E2M1>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  using Sh = RowsShape<D, E2M1>;
  constexpr int kSmem = Sh::kBytes + 1024;
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> ready[kMaxDevices];
  int sms = 0, dev = 0;
  cudaError_t e = attn_sm_count(&sms);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_attn_rows<D, E2M1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
  }
  CUtensorMap k_map, v_map;
  e = attn_code_map(&k_map, a, a.k_codes, Sh::kRowBytes, true);
  if (e == cudaSuccess) e = attn_code_map(&v_map, a, a.v_codes, Sh::kRowBytes, true);
  if (e != cudaSuccess) return e;
  k_attn_rows<D, E2M1><<<sms * kCtasPerSm < kAttnMaxCtas ? sms * kCtasPerSm : kAttnMaxCtas, kThreads, kSmem, s>>>(a, k_map, v_map);
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
