// Reading MX cache elements: E4M3 and E2M1 pairs to f16 (both are exact there)
// and E8M0 scales; a token's place in a paged cache.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace mxk {

// Two E4M3 codes (low byte first) as f16x2.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Two E2M1 codes (one byte, low nibble first) as f16x2.
__device__ __forceinline__ uint32_t f16x2_of_e2m1x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "mov.b16 {b0, b1}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// 2^(code - 127) as fp32 (code 0 is the subnormal 2^-127, 255 is NaN).
__device__ __forceinline__ float e8m0_value(int code) {
  return __uint_as_float(code > 0 && code < 255 ? static_cast<uint32_t>(code) << 23 : code == 0 ? 1u << 22 : 0x7FC00000u);
}

// Cache row (page, place) of token t: the sequence that holds it by a 32-way
// search of q_starts, its position counted back from the sequence's length.
// Returns the row index (page * n_kv_heads) * page_size + place of head 0, or
// -1 for a token past the last sequence; bad metadata sets the status word.
// `pos` gets the token's position (where there is one).
__device__ __forceinline__ int64_t token_row(const KvArgs& a, int t, int lane, int64_t& pos) {
  int lo = 0, hi = a.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && a.q_starts[i] <= t;
    const int n = max(__popc(__ballot_sync(0xffffffffu, le)), 1);
    lo += (n - 1) * step;
    hi = min(lo + step, hi);
  }
  const int start = a.q_starts[lo], end = a.q_starts[lo + 1], kv = a.kv_lens[lo];
  if (t >= end) return -1;
  pos = static_cast<int64_t>(kv) - (end - t);
  if (start < 0 || start > t || end > a.T || pos < 0 || kv > static_cast<int64_t>(a.max_pages) * a.page_size) {
    if (lane == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
    return -1;
  }
  const int p = static_cast<int>(pos) / a.page_size;  // positions are ints: kv has been checked
  const int page = a.block_table[static_cast<int64_t>(lo) * a.max_pages + p];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) set_status(a.status, MX_ERR_DEVICE_ARG);
    return -1;
  }
  return static_cast<int64_t>(page) * a.n_heads * a.page_size + (pos - static_cast<int64_t>(p) * a.page_size);
}

}  // namespace mxk
