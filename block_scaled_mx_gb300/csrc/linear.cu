// Dense products with MX weights: out[t, n] = bias[n] + sum_k A[t, k] W[n, k] for MX
// activations A (E4M3 or E2M1) and MX weights W, as block-scaled tcgen05 MMAs with fp32
// accumulators in tensor memory.
//
// Weights are the MMA's A operand (128 rows of N a block), tokens its B operand (`bn` of
// them a tile), so a decoding step of a few tokens still runs full-width MMAs while the
// weights stream.  All operands come by TMA, the scales too: they lie in 512-byte blocks
// of 128 rows x 4 scales in the order that tcgen05.cp copies to tensor memory, the
// weights' laid out once (mx_linear_prepare), the tokens' by a first launch, which also
// quantises bf16 activations.  The MMAs' launch is a dependent one: its set-up and its
// first weights come while the first launch runs.
//
// Warps: 0 TMA, 1 tensor memory and MMAs (one thread), 2..9 epilogue (two to a quarter of
// tensor memory's lanes).  Accumulators are double-buffered where tensor memory holds
// two.  Three forms:
//   split  clusters of S CTAs share a tile's K; the parts are added in rank order
//          through distributed shared memory (the same bits every time)
//   whole  a CTA goes through tiles of all of K
//   pair   two CTAs share a 256-row tile: cta_group::2 MMAs, each loads half the tokens
// Every wait is bounded; one that runs out sets MX_ERR_TIMEOUT and all roles unwind.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace mxk {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kMaxStages = 12;
constexpr int kBand = 8;

struct Params {
  int T, N, RB, TT, KS;  // KS: stages of all of K (128 bytes of every row each)
  int bn, brows;         // tokens of a tile, of this CTA's loads (half in a pair)
  int splits, units;     // CTAs that share a tile's K; tiles (of pairs in a pair)
  int stages, acc_bufs;
  int a_fmt, out_f32, slice, half_blocks;  // half_blocks: a stage is half of a weight block (E2M1 widened to bytes)
  uint32_t a_tx;         // bytes that a stage's weights count for
  uint32_t b_slot;       // shared memory of a stage's tokens
  uint32_t off_b, off_sa, off_sb, off_bar;
  uint32_t tmem_cols, acc_cols, sf_col0;
  const float* bias;
  void* out;
  int* status;
  unsigned long long wait_limit_ns;
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
};

template <bool PAIR>
struct Waiter {
  Bars* b;
  uint32_t peer_abort;  // the peer's flag in a pair
  unsigned long long limit_ns;
  int* status;
  __device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, bool sleep) const {
    if (PAIR) return sleep ? mbar_try_wait_cluster_sleep(bar, parity, 20000u) : mbar_try_wait_cluster(bar, parity);
    return sleep ? mbar_try_wait_sleep(bar, parity, 20000u) : mbar_try_wait(bar, parity);
  }
  // False when the wait ran out or another role gave up.
  __device__ __forceinline__ bool operator()(uint64_t* bar64, uint32_t parity, bool sleep = true) const {
    const uint32_t bar = smem_u32(bar64);
    if (poll(bar, parity, false)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
      if (poll(bar, parity, sleep)) return true;
      if (*static_cast<volatile int*>(&b->abort)) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        set_status(status, MX_ERR_TIMEOUT);
        *static_cast<volatile int*>(&b->abort) = 1;
        if (PAIR) st_shared_cluster_u32(peer_abort, 1u);
        return false;
      }
    }
  }
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity)) != 0;
  }
};

__device__ __forceinline__ void store_out(const Params& p, int64_t at, float v) {
  if (p.out_f32) static_cast<float*>(p.out)[at] = v;
  else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// A4: both operands packed E2M1 (kind::mxf4, 256 elements a stage), else kind::mxf8f6f4
// (128 elements; E2M1 weights are widened to bytes by the TMA).  NSB: blocks of 128 tokens
// that a tile touches.
template <bool PAIR, bool A4, int NSB>
__global__ void __launch_bounds__(kThreads, PAIR ? 1 : 2)
    k_linear(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
             const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Bars* const bars = reinterpret_cast<Bars*>(base + p.off_bar);
  constexpr int kSub = A4 ? 2 : 1;                      // scale blocks of a stage along K
  constexpr uint32_t kSa = kSub * 512u, kSb = NSB * kSub * 512u;
  constexpr uint32_t kSfCols = 4u + 4u * NSB;           // tensor-memory columns of a scale block's set
  const int S = p.stages;
  const uint32_t rank = PAIR || p.splits > 1 ? cluster_ctarank() : 0u;
  const int group = PAIR ? 2 : p.splits;
  const int unit0 = blockIdx.x / group, unit_step = gridDim.x / group;
  const int k0 = PAIR ? 0 : static_cast<int>(static_cast<int64_t>(p.KS) * rank / p.splits);
  const int k1 = PAIR ? p.KS : static_cast<int>(static_cast<int64_t>(p.KS) * (rank + 1) / p.splits);
  const int rbs = PAIR ? (p.RB + 1) / 2 : p.RB;  // tiles along N
  // Tile of a unit: bands of kBand tiles along N, each through all tokens, so that the
  // CTAs at work share both operands' rows.
  auto tile_of = [&](int unit, int& tt, int& rb) {
    const int band = unit / (kBand * p.TT), in = unit - band * kBand * p.TT, wide = min(kBand, rbs - band * kBand);
    tt = in / wide;
    rb = band * kBand + in - tt * wide;
    if (PAIR) rb = 2 * rb + static_cast<int>(rank);
  };

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), PAIR ? 2 : 1);  // one arrival with bytes from each CTA's TMA warp
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&bars->acc_full[a]), 1);
      mbar_init(smem_u32(&bars->acc_empty[a]), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(&bars->tmem), p.tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&bars->tmem), p.tmem_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // barriers are ready before the peer arrives on them
  tc_fence_after();
  const uint32_t tbase = bars->tmem;
  const Waiter<PAIR> wait{bars, PAIR ? mapa_shared(smem_u32(&bars->abort), rank ^ 1u) : 0u, p.wait_limit_ns, p.status};

  if (warp == 0) {
    // ================================================================ TMA
    if (elect_one()) {
      // A single thread feeds the MMAs, so what it does for a stage is MMA time: all that
      // does not change from stage to stage is worked out once a tile.
      uint32_t fills = 0, s = 0, ph = 0;
      bool ok = true, ready = false;
      const uint32_t full0 = smem_u32(bars->full), a0 = smem_u32(base);
      const uint32_t b0 = a0 + p.off_b, sa0 = a0 + p.off_sa, sb0 = a0 + p.off_sb, b_slot = p.b_slot;
      const uint32_t bar0 = PAIR ? mapa_shared(full0, 0u) : full0;  // in a pair all copies land on rank 0's barriers
      const uint32_t bytes = p.a_tx + static_cast<uint32_t>(p.brows) * 128u + kSa + kSb;
      const int units = p.units;
      const bool half_blocks = p.half_blocks != 0;
      int tt, rb = 0, row0 = 0, tb0 = 0;  // of the tile
      // weights of one stage; its barrier is armed for everything that lands there
      auto weights = [&](uint32_t slot, int k) {
        const uint32_t bar = bar0 + slot * 8u, a = a0 + slot * 16384u, sa = sa0 + slot * kSa;
        const int x = half_blocks ? (k & 1) * 128 : 0, kb = half_blocks ? k >> 1 : k;
        if (PAIR) {
          mbar_arrive_expect_tx_cluster_relaxed(bar, bytes);
          tma_load_4d_pair(a, &tm_a, x, 0, kb, rb, bar);
          tma_load_3d_pair(sa, &tm_sa, 0, k * kSub, rb, bar);
        } else {
          mbar_arrive_expect_tx(bar, bytes);
          tma_load_4d(a, &tm_a, x, 0, kb, rb, bar);
          tma_load_3d(sa, &tm_sa, 0, k * kSub, rb, bar);
        }
      };
      auto tokens = [&](uint32_t slot, int k) {
        const uint32_t bar = bar0 + slot * 8u, b = b0 + slot * b_slot, sb = sb0 + slot * kSb;
        if (PAIR) {
          tma_load_2d_pair(b, &tm_b, k * 128, row0, bar);
          tma_load_3d_pair(sb, &tm_sb, 0, k * kSub, tb0, bar);
        } else {
          tma_load_2d(b, &tm_b, k * 128, row0, bar);
          tma_load_3d(sb, &tm_sb, 0, k * kSub, tb0, bar);
        }
      };
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_sa);
      prefetch_tensormap(&tm_b);
      prefetch_tensormap(&tm_sb);
      for (int unit = unit0; unit < units && ok; unit += unit_step) {
        tile_of(unit, tt, rb);
        tb0 = tt * p.bn / 128;
        row0 = tt * p.bn + (PAIR ? static_cast<int>(rank) * p.brows : 0);
        int k = k0;
        if (!ready) {
          // the first launch's results are awaited behind the weights of all stages
          int n = 0;
          for (; n < S && k0 + n < k1; ++n) weights(n, k0 + n);
          asm volatile("griddepcontrol.wait;" ::: "memory");
          ready = true;
          for (int i = 0; i < n; ++i) tokens(i, k++);
          fills = n;
          s = n % S;
          ph = n / S;
        }
        for (; k < k1; ++k) {
          if (!wait(&bars->empty[s], ph ^ 1u)) {
            ok = false;
            break;
          }
          weights(s, k);
          tokens(s, k);
          ++fills;
          if (++s == static_cast<uint32_t>(S)) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // what this thread asked for has landed before the CTA leaves (in a pair rank 0's
      // barriers count both CTAs' copies)
      if (!PAIR || rank == 0) {
        for (int i = 0; i < S && static_cast<uint32_t>(i) < fills; ++i) {
          const uint32_t last = fills - 1 - ((fills - 1 - i) % S);
          mbar_wait(smem_u32(&bars->full[i]), (last / S) & 1u, 100000000ull);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ MMAs
    if ((!PAIR || rank == 0) && elect_one()) {
      const uint32_t smem0 = smem_u32(base);
      const uint32_t a0 = desc_lo_sw128(smem0), b0 = desc_lo_sw128(smem0 + p.off_b), b_step = p.b_slot >> 4;
      const uint32_t sa0 = scales_desc_lo(smem0 + p.off_sa), sb0 = scales_desc_lo(smem0 + p.off_sb);
      const uint32_t sf0 = tbase + p.sf_col0, sf_end = sf0 + 4u * kSfCols;  // four sets of scale columns in turn
      const int units = p.units, bn = p.bn, T = p.T;
      constexpr uint32_t kM = PAIR ? 256u : 128u;
      uint32_t s = 0, ph = 0, ab = 0, aph = 0, sf = sf0;
      uint32_t a = a0, b = b0, sa = sa0, sb = sb0;
      bool ok = true;
      for (int unit = unit0; unit < units && ok; unit += unit_step) {
        int tt, rb;
        tile_of(unit, tt, rb);
        const int n0 = tt * bn;
        const uint32_t sb_col = 4u + static_cast<uint32_t>(n0 % 128) / 32;
        // a pair's CTAs hold the two halves of a whole tile
        const uint32_t n_mma = static_cast<uint32_t>(PAIR ? bn : (min(bn, T - n0) + 15) & ~15);
        uint32_t idesc[A4 ? 2 : 4];
#pragma unroll
        for (int i = 0; i < (A4 ? 2 : 4); ++i)
          idesc[i] = A4 ? idesc_mxf4(kM, n_mma, 2 * i) : idesc_mx(p.a_fmt, kFmtE4M3, kM, n_mma, i, i);
        if (!wait(&bars->acc_empty[ab], aph ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tbase + ab * p.acc_cols;
        for (int k = k0; k < k1; ++k) {
          if (!wait(&bars->full[s], ph, false)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t accum = k > k0;
#pragma unroll
          for (int c = 0; c < kSub; ++c) {
            if (PAIR) tmem_copy_scales_pair(sf + c * kSfCols, sa + c * 32u);
            else tmem_copy_scales_lo(sf + c * kSfCols, sa + c * 32u);
#pragma unroll
            for (int i = 0; i < NSB; ++i) {
              if (PAIR) tmem_copy_scales_pair(sf + c * kSfCols + 4u + 4u * i, sb + (i * kSub + c) * 32u);
              else tmem_copy_scales_lo(sf + c * kSfCols + 4u + 4u * i, sb + (i * kSub + c) * 32u);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f = sf + (A4 ? i / 2 : 0) * kSfCols;
            if (A4) {
              if (PAIR) mma_mxf4_pair_lo(d, a + 2u * i, b + 2u * i, kDescHiSw128, idesc[i & 1], f, f + sb_col, i ? 1u : accum);
              else mma_mxf4_lo(d, a + 2u * i, b + 2u * i, kDescHiSw128, idesc[i & 1], f, f + sb_col, i ? 1u : accum);
            } else {
              if (PAIR) mma_mxf8f6f4_pair_lo(d, a + 2u * i, b + 2u * i, kDescHiSw128, idesc[A4 ? 0 : i], f, f + sb_col, i ? 1u : accum);
              else mma_mxf8f6f4_lo(d, a + 2u * i, b + 2u * i, kDescHiSw128, idesc[A4 ? 0 : i], f, f + sb_col, i ? 1u : accum);
            }
          }
          if (PAIR) mma_commit_pair(smem_u32(&bars->empty[s]), 3);
          else mma_commit(smem_u32(&bars->empty[s]));
          sf += kSub * kSfCols;
          if (sf == sf_end) sf = sf0;
          a += 16384u >> 4;
          b += b_step;
          sa += kSa >> 4;
          sb += kSb >> 4;
          if (++s == static_cast<uint32_t>(S)) {
            s = 0;
            ph ^= 1u;
            a = a0;
            b = b0;
            sa = sa0;
            sb = sb0;
          }
        }
        if (!ok) break;
        if (PAIR) mma_commit_pair(smem_u32(&bars->acc_full[ab]), 3);
        else mma_commit(smem_u32(&bars->acc_full[ab]));
        if (++ab == static_cast<uint32_t>(p.acc_bufs)) {
          ab = 0;
          aph ^= 1u;
        }
      }
      // every MMA has completed before tensor memory is given back
      if (PAIR) mma_commit_pair(smem_u32(&bars->drain), 1);
      else mma_commit(smem_u32(&bars->drain));
      mbar_wait(smem_u32(&bars->drain), 0, 100000000ull);
    }
    __syncwarp();
  } else if (PAIR || p.splits == 1) {
    // ================================================================ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint32_t ab = 0, aph = 0;
    for (int unit = unit0; unit < p.units; unit += unit_step) {
      int tt, rb;
      tile_of(unit, tt, rb);
      const int n0 = tt * p.bn, cols = min(p.bn, p.T - n0);
      const int n = rb * 128 + 32 * q + lane;
      const float bias = p.bias && n < p.N ? __ldg(p.bias + n) : 0.0f;
      if (!wait.warp(&bars->acc_full[ab], aph)) break;
      tc_fence_after();
      const uint32_t d = tbase + (static_cast<uint32_t>(32 * q) << 16) + ab * p.acc_cols;
      for (int c0 = 32 * half; c0 < cols; c0 += 64) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(d + c0, r);
        tmem_ld_wait();
        const int64_t at = static_cast<int64_t>(n0 + c0) * p.N + n;
        if (!p.out_f32 && p.N % 2 == 0) {
          // two lanes exchange a token each, so that a lane stores two neighbours of one
          const bool odd = lane & 1;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float v0 = __uint_as_float(r[c]) + bias, v1 = __uint_as_float(r[c + 1]) + bias;
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(other, v1) : __floats2bfloat162_rn(v0, other);
            if (c0 + c + odd < cols && n < p.N)
              *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at + static_cast<int64_t>(c + odd) * p.N - odd) = w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < cols && n < p.N) store_out(p, at + static_cast<int64_t>(c) * p.N, __uint_as_float(r[c]) + bias);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&bars->acc_empty[ab]), 0u));
        else mbar_arrive(smem_u32(&bars->acc_empty[ab]));
      }
      if (++ab == static_cast<uint32_t>(p.acc_bufs)) {
        ab = 0;
        aph ^= 1u;
      }
    }
  } else {
    // split: one tile a cluster; its parts are added below
    wait.warp(&bars->acc_full[0], 0);
    tc_fence_after();
  }

  if (!PAIR && p.splits > 1) {
    // Rank r adds up columns [r * slice, (r + 1) * slice) of the tile: every CTA stores its
    // part of them in r's shared memory (the stages', which all CTAs have read by now).
    __syncthreads();
    cluster_sync_all();
    float* const parts = reinterpret_cast<float*>(base);  // [source][128 rows][pitch]
    const int slice = p.slice, pitch = slice + 4;                   // rows 16 bytes apart modulo 128: no bank conflicts
    int tt, rb;
    tile_of(unit0, tt, rb);
    const int n0 = tt * p.bn, cols = min(p.bn, p.T - n0);
    if (warp >= 2) {
      const int q = warp & 3, half = (warp - 2) >> 2;
      const uint32_t d = tbase + (static_cast<uint32_t>(32 * q) << 16);
      const uint32_t mine = smem_u32(parts + (static_cast<int>(rank) * 128 + 32 * q + lane) * pitch);
      for (int c0 = 8 * half; c0 < cols; c0 += 16) {
        uint32_t r[8];
        __syncwarp();
        tmem_ld_32x32b_x8(d + c0, r);
        const int owner = c0 / slice;  // eight columns have one: slice is a multiple of eight
        const uint32_t at = mapa_shared(mine + static_cast<uint32_t>(c0 - owner * slice) * 4u, static_cast<uint32_t>(owner));
        tmem_ld_wait();
        st_shared_cluster_v4(at, r[0], r[1], r[2], r[3]);
        st_shared_cluster_v4(at + 16u, r[4], r[5], r[6], r[7]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    const int first = static_cast<int>(rank) * slice, left = min(slice, cols - first);
    if (!bars->abort) {
      for (int i = tid; i < 128 * ((left + 3) / 4); i += kThreads) {
        const int row = i & 127, c0 = (i >> 7) * 4, n = rb * 128 + row;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < p.splits; ++s) {
          const float4 w = *reinterpret_cast<const float4*>(parts + (s * 128 + row) * pitch + c0);
          v[0] += w.x;
          v[1] += w.y;
          v[2] += w.z;
          v[3] += w.w;
        }
        if (n < p.N) {
          const float bias = p.bias ? __ldg(p.bias + n) : 0.0f;
          const int64_t at = static_cast<int64_t>(n0 + first + c0) * p.N + n;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c0 + c < left) store_out(p, at + static_cast<int64_t>(c) * p.N, v[c] + bias);
        }
      }
    }
  }
  tc_fence_before();
  // One answer for the whole CTA: the peer may still set the flag (it does so ahead of the
  // cluster's barrier below), and threads that read it for themselves would part here.
  if (__syncthreads_or(PAIR && *static_cast<volatile int*>(&bars->abort))) {
    // where a wait ran out nobody counts rank 1's last copies: they get a millisecond
    if (tid == 0) {
      for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000ull;) {
      }
    }
    __syncthreads();
  }
  if (PAIR) cluster_sync_all();  // neither leaves while the other's MMAs or copies may reach it
  tc_fence_after();
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tbase, p.tmem_cols);
    else tmem_dealloc(tbase, p.tmem_cols);
  }
}

// ------------------------------------------------------------------ tokens
// bf16 rows to MX codes and tiled scales, or (x null) row-major scales to tiled ones.  A
// lane has eight elements, four lanes a block of 32; scale blocks behind K are 1.
// Tiled: block (t / 128, k / 128) of 512 bytes, word [t % 32][t % 128 / 32] its row's four.
// Memory-bound: four 16-byte loads a thread are on their way before the first is used, a
// warp goes through neighbouring groups and counts its place on, and a block's largest
// magnitude is found on the bf16 words (8192 x 4096 to MXFP4: 30 us with divisions and one
// load at a time, 23 so, with the ALU pipe at 77%; the bytes at copy rate: 12.6).
constexpr int kTokenUnroll = 4;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  asm("max.u16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}

// Byte of a token's scale of its first block among the tiled ones; block b (of 32 elements)
// is at + b / 4 * 512 + b % 4.
__device__ __forceinline__ size_t tiled_row(int t, int NK) {
  return static_cast<size_t>(t / 128) * NK * 512 + (t % 32) * 16 + (t % 128 / 32) * 4;
}

template <bool E2M1>
__global__ void __launch_bounds__(256) k_linear_tokens(const uint4* __restrict__ x, const uint8_t* __restrict__ scales, int t0, int n, int K, int NK,
                                                       FastDiv per_row_div, uint8_t* __restrict__ codes, uint8_t* __restrict__ tiled) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!x) {  // n scales, per_row of a token
    const int per_row = NK * 4;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
      const int r = per_row_div.of(i), b = i - r * per_row, t = t0 + r;
      tiled[tiled_row(t, NK) + b / 4 * 512 + b % 4] = b < K / 32 ? scales[static_cast<size_t>(t) * (K / 32) + b] : 127;
    }
    return;
  }
  const int per_row = NK * 16, k8 = K / 8;  // n groups of eight, per_row of a token
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * (32 * kTokenUnroll) + lane;
  if (i0 - lane >= n) return;
  int t[kTokenUnroll], g[kTokenUnroll];
  t[0] = per_row_div.of(i0);
  g[0] = i0 - t[0] * per_row;
  t[0] += t0;
  uint4 w[kTokenUnroll];
#pragma unroll
  for (int u = 0; u < kTokenUnroll; ++u) {
    if (u > 0) {
      t[u] = t[u - 1];
      g[u] = g[u - 1] + 32;
      while (g[u] >= per_row) {
        g[u] -= per_row;
        ++t[u];
      }
    }
    w[u] = i0 + u * 32 < n && g[u] < k8 ? __ldcs(x + static_cast<int64_t>(t[u]) * k8 + g[u]) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kTokenUnroll; ++u) {
    if (i0 - lane + u * 32 >= n) break;
    const uint32_t b[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    constexpr uint32_t kSize = 0x7FFF7FFFu;
    const uint32_t m = max_u16x2(max_u16x2(b[0] & kSize, b[1] & kSize), max_u16x2(b[2] & kSize, b[3] & kSize));
    uint32_t amax = max(m & 0xFFFFu, m >> 16);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int s = mx_block_exponent(amax << 16, E2M1 ? 2 : 8);
    const float p = pow2_neg(s);
    const bool here = i0 + u * 32 < n, in = here && g[u] < k8;
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(b[i] << 16) * p, hi = __uint_as_float(b[i] & 0xFFFF0000u) * p;
      if (E2M1) c[0] |= enc_e2m1x2(lo, hi) << (8 * i);
      else c[i / 2] |= enc_e4m3x2(lo, hi) << (16 * (i % 2));
    }
    if (in) {
      const int64_t at = static_cast<int64_t>(t[u]) * k8 + g[u];
      if (E2M1) reinterpret_cast<uint32_t*>(codes)[at] = c[0];
      else reinterpret_cast<uint2*>(codes)[at] = make_uint2(c[0], c[1]);
    }
    if (here && (g[u] & 3) == 0) tiled[tiled_row(t[u], NK) + (g[u] >> 4) * 512 + (g[u] >> 2) % 4] = in ? static_cast<uint8_t>(s + 127) : 127;
  }
}

// Weights to blocks of 128 rows x 128 bytes and their scales to tiled ones; rows
// behind N and elements behind K are zeros of scale 1.
__global__ void __launch_bounds__(256) k_linear_prepare(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, LinearLayout L,
                                                        uint8_t* __restrict__ dst) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x, i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  constexpr int row16 = 8;                                          // 16-byte pieces of a block's row
  const int src16 = (L.e2m1 ? L.K / 2 : L.K) / 16;                  // of a weight's row
  const int64_t blocks = static_cast<int64_t>(L.RB) * L.NB, pieces = blocks * 128 * row16;
  for (int64_t i = i0; i < pieces; i += stride) {
    const int64_t b = i / (128 * row16);
    const int in = static_cast<int>(i - b * (128 * row16)), r = in / row16, c = in - r * row16;
    const int rb = static_cast<int>(b / L.NB), kc = static_cast<int>(b - static_cast<int64_t>(rb) * L.NB);
    const int64_t n = static_cast<int64_t>(rb) * 128 + r;
    const int k = kc * row16 + c;
    reinterpret_cast<uint4*>(dst)[i] = n < L.N && k < src16 ? __ldg(reinterpret_cast<const uint4*>(codes) + n * src16 + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  for (int64_t i = i0; i < static_cast<int64_t>(L.RB) * L.NK * 512; i += stride) {
    const int64_t b = i / 512;
    const int in = static_cast<int>(i - b * 512);
    const int rb = static_cast<int>(b / L.NK), kc = static_cast<int>(b - static_cast<int64_t>(rb) * L.NK);
    const int64_t n = static_cast<int64_t>(rb) * 128 + (in / 4 % 4) * 32 + in / 16;
    const int k = kc * 4 + in % 4;
    dst[L.scales_offset + i] = n < L.N && k < L.K / 32 ? scales[n * (L.K / 32) + k] : 127;
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

constexpr uint32_t kSmem = 227 * 1024;

// Shared and tensor memory of a form; false where it does not fit.
bool lay_out(Params& p, bool pair, bool a4, int nsb, uint32_t budget, uint32_t* smem) {
  const uint32_t sa = a4 ? 1024u : 512u, sb = sa * nsb, sf_cols = 4u + 4u * nsb;
  p.brows = pair ? p.bn / 2 : p.bn;
  p.b_slot = static_cast<uint32_t>(p.brows) * 128u;
  p.acc_cols = static_cast<uint32_t>(p.bn + 31) & ~31u;
  p.acc_bufs = p.splits == 1 && 2 * p.acc_cols + 4 * sf_cols <= 512 ? 2 : 1;
  p.sf_col0 = p.acc_bufs * p.acc_cols;
  const uint32_t cols = p.sf_col0 + 4 * sf_cols;
  if (cols > 512) return false;
  for (p.tmem_cols = 32; p.tmem_cols < cols;) p.tmem_cols *= 2;
  const uint32_t stage = 16384u + p.b_slot + sa + sb;
  const uint32_t fixed = 1024u + static_cast<uint32_t>((sizeof(Bars) + 127) & ~size_t(127));
  p.stages = std::min<int>(kMaxStages, static_cast<int>((budget - fixed) / stage));
  if (p.stages < 2) return false;
  const uint32_t n = static_cast<uint32_t>(p.stages);
  p.off_b = n * 16384u;
  p.off_sa = p.off_b + n * p.b_slot;
  p.off_sb = p.off_sa + n * sa;
  p.off_bar = p.off_sb + n * sb;
  *smem = p.off_bar + fixed;
  p.slice = ((p.bn + p.splits - 1) / p.splits + 7) & ~7;
  // the parts of a split tile lie where the stages were
  return p.splits == 1 || static_cast<uint32_t>(p.splits * (p.slice + 4)) * 512u <= p.off_bar;
}

struct Form {
  bool pair, half;  // half: two CTAs share an SM
  int bn, splits;
};

// Which form a call takes, by sizes.  A call's time is its weights' stream and a start of
// some 6 us; in us, MXFP8 on both sides, K -> N:
//   few tokens: two CTAs an SM, K split so that some 200 CTAs stream (a cluster of three
//     with an SM to each CTA leaves SMs that no cluster fits)
//       1 token, 4096 -> 6144      whole 12.4, split in 2 / 3 / 4 / 5: 11.9 / 11.8 / 11.1 / 11.4
//       1 token, 4096 -> 20000     whole with an SM to each CTA 24.4, two an SM 19.5
//   more: pairs, whose wave of tiles takes about 94 + bn
//       96 tokens, 4096 -> 6144    pair 13.0, split in 2: 15.4    160: 13.5 and 17
//       700 tokens, 4096 -> 6144   bn 64 / 128 / 192: 32.5 / 24.0 / 26.2
//       700 tokens, 4096 -> 20000  75 / 51.8 / 48.8
//   but a long K over few tiles is split all the same
//       96 tokens, 16384 -> 4096   pair 27, tiles of 64 tokens split in 4: 24.6
Form choose_form(int T, int RB, int KS) {
  const int rbs = (RB + 1) / 2;
  auto split = [&](int bn) {
    const int tiles = RB * ((T + bn - 1) / bn);
    Form f{false, true, bn, 1};
    while (f.splits < 8 && tiles * (f.splits + 1) <= 228 && KS / (f.splits + 1) >= 4) ++f.splits;
    return f;
  };
  if (T <= 32 || (T <= 64 && RB <= 24)) return split((T + 15) & ~15);
  if (T <= 256 && KS >= 64 && rbs * ((T + 63) / 64) <= 38) return split(64);
  Form best{true, false, 64, 1};
  int64_t least = INT64_MAX;
  for (int bn = 64; bn <= 192; bn += 64) {
    const int64_t waves = (static_cast<int64_t>((T + bn - 1) / bn) * rbs + 75) / 76, time = waves * (94 + bn);
    if (time < least) {
      least = time;
      best.bn = bn;
    }
  }
  return best;
}

using Kernel = void (*)(Params, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap);
Kernel kernel_of(bool pair, bool a4, int nsb) {
  if (pair && nsb == 1) return a4 ? k_linear<true, true, 1> : k_linear<true, false, 1>;
  if (pair) return a4 ? k_linear<true, true, 2> : k_linear<true, false, 2>;
  return a4 ? k_linear<false, true, 1> : k_linear<false, false, 1>;  // at most 64 tokens a tile
}

}  // namespace

LinearLayout linear_layout(int N, int K, int fmt) {
  LinearLayout L{};
  L.N = N;
  L.K = K;
  L.e2m1 = fmt == MX_E2M1;
  L.RB = (N + 127) / 128;
  L.NB = L.e2m1 ? (K + 255) / 256 : (K + 127) / 128;
  L.NK = L.e2m1 ? 2 * L.NB : L.NB;
  L.scales_offset = static_cast<size_t>(L.RB) * L.NB * 16384;
  L.total_bytes = L.scales_offset + static_cast<size_t>(L.RB) * L.NK * 512;
  return L;
}

cudaError_t launch_linear_prepare(const uint8_t* codes, const uint8_t* scales, const LinearLayout& L, uint8_t* dst, cudaStream_t s) {
  const int64_t pieces = static_cast<int64_t>(L.scales_offset) / 16;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((pieces + 255) / 256, 152 * 8));
  k_linear_prepare<<<grid, 256, 0, s>>>(codes, scales, L, dst);
  return cudaGetLastError();
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  auto encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  const LinearLayout L = linear_layout(a.N, a.K, a.w_fmt);
  const bool a4 = a.act_fmt == MX_E2M1;
  const int TB = (a.T + 127) / 128;
  Params p{};
  p.T = a.T;
  p.N = a.N;
  p.RB = L.RB;
  p.KS = a4 ? L.NB : (a.K + 127) / 128;
  p.a_fmt = a.w_fmt == MX_E4M3 ? kFmtE4M3 : kFmtE2M1;
  p.half_blocks = a.w_fmt == MX_E2M1 && !a4;
  p.a_tx = p.half_blocks ? 8192u : 16384u;
  p.out_f32 = a.out_f32;
  p.bias = a.bias;
  p.out = a.out;
  p.status = a.status;
  p.wait_limit_ns = a.wait_limit_ns;

  const Form f = choose_form(a.T, p.RB, p.KS);
  const bool pair = f.pair;
  p.bn = f.bn;
  p.splits = f.splits;
  p.TT = (a.T + p.bn - 1) / p.bn;
  p.units = p.TT * (pair ? (p.RB + 1) / 2 : p.RB);
  // token tiles start at multiples of 64 of their blocks of 128
  const int nsb = p.TT == 1 ? (p.bn + 127) / 128 : p.bn % 128 == 0 || p.bn == 64 ? (p.bn + 127) / 128 : p.bn / 128 + 1;
  uint32_t smem = 0;
  if (!(f.half && lay_out(p, pair, a4, nsb, kSmem / 2 - 1024, &smem)) && !lay_out(p, pair, a4, nsb, kSmem, &smem)) return cudaErrorInvalidConfiguration;
  const int fit = 152 * (f.half ? 2 : 1);
  const uint32_t ctas = p.splits > 1 ? p.units * p.splits : pair ? 2 * std::min(p.units, fit / 2) : std::min(p.units, fit);

  CUtensorMap tm_a, tm_b, tm_sa, tm_sb;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  {
    // blocks of 128 rows x 128 bytes; as elements where E2M1 is widened
    const cuuint64_t inner = p.half_blocks ? 256 : 128;
    const cuuint64_t dims[4] = {inner, 128, static_cast<cuuint64_t>(L.NB), static_cast<cuuint64_t>(L.RB)};
    const cuuint64_t strides[3] = {128, 16384, 16384 * static_cast<cuuint64_t>(L.NB)};
    const cuuint32_t box[4] = {128, 128, 1, 1};
    if (encode(&tm_a, p.half_blocks ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(a.w_prep), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t row = static_cast<cuuint64_t>(a4 ? a.K / 2 : a.K);
    const cuuint64_t dims[2] = {row, static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[1] = {row};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(p.brows)};
    if (encode(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.t_codes), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    // scales as [block of 128 rows][scale block along K][128 words]
    const uint8_t* src = i ? a.t_scales : a.w_prep + L.scales_offset;
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(L.NK), static_cast<cuuint64_t>(i ? TB : L.RB)};
    const cuuint64_t strides[2] = {512, 512 * static_cast<cuuint64_t>(L.NK)};
    const cuuint32_t box[3] = {128, a4 ? 2u : 1u, i ? static_cast<cuuint32_t>(nsb) : 1u};
    if (encode(i ? &tm_sb : &tm_sa, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(src), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }

  {
    const int per_row = L.NK * (a.x ? 16 : 4);
    const int most = (1 << 30) / per_row;  // tokens of a launch: places are ints
    for (int t0 = 0; t0 < a.T; t0 += most) {
      const int n = std::min(most, a.T - t0) * per_row;
      const unsigned grid = a.x ? static_cast<unsigned>((n + 256 * kTokenUnroll - 1) / (256 * kTokenUnroll)) : static_cast<unsigned>(std::min((n + 255) / 256, 152 * 8));
      const uint4* x = static_cast<const uint4*>(a.x);
      uint8_t* codes = const_cast<uint8_t*>(a.t_codes);
      const FastDiv div = FastDiv::by(per_row);
      if (a4) k_linear_tokens<true><<<grid, 256, 0, s>>>(x, a.scales, t0, n, a.K, L.NK, div, codes, a.t_scales);
      else k_linear_tokens<false><<<grid, 256, 0, s>>>(x, a.scales, t0, n, a.K, L.NK, div, codes, a.t_scales);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  const Kernel kernel = kernel_of(pair, a4, nsb);
  static std::atomic<uint64_t> allowed[6];
  cudaError_t e = allow_smem(kernel, allowed[(pair ? nsb : 0) * 2 + a4], static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = pair ? 2 : p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, tm_a, tm_b, tm_sa, tm_sb);
}

}  // namespace mxk
