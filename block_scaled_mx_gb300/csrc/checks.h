// Argument checks that several calls of the C ABI share.
#pragma once
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "../../include/mxmoe.h"
#include "internal.h"

namespace mxk {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }
inline bool type_ok(int t) { return t == MX_BF16 || t == MX_F32; }
inline bool finite_positive(float v) { return v > 0.0f && v <= 3.402823466e38f; }

// The cache and the batch's sizes, as the cache calls take them.
inline int check_cache(const mx_kv_cache* c, int n_seqs, int max_pages, int T) {
  if (!c || T < 0 || n_seqs < 0 || max_pages <= 0) return MX_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0) return MX_ERR_INVALID_ARG;
  if (c->fmt != MX_E4M3 && c->fmt != MX_E2M1) return MX_ERR_INVALID_ARG;
  if (c->head_dim % 32) return MX_ERR_UNSUPPORTED;
  // positions, heads x elements and grid sizes are ints
  if (static_cast<int64_t>(max_pages) * c->page_size > INT_MAX / 2) return MX_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->n_kv_heads) * c->head_dim > (1 << 20) || T > INT_MAX / 2) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

inline int check_cache_pointers(const mx_kv_cache* c, const void* block_table, const void* kv_lens, const void* q_starts,
                         const void* ws, size_t ws_bytes) {
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !block_table || !kv_lens || !q_starts || !ws)
    return MX_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16) ||
      !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_starts, 4) || !aligned(ws, 256))
    return MX_ERR_ALIGNMENT;
  return ws_bytes < 256 ? MX_ERR_WORKSPACE : MX_OK;
}

inline KvArgs kv_args(const mx_kv_cache* c, const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts,
               int n_seqs, int max_pages, int T, void* ws) {
  KvArgs a{};
  a.k_codes = c->k_codes;
  a.k_scales = c->k_scales;
  a.v_codes = c->v_codes;
  a.v_scales = c->v_scales;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.n_heads = c->n_kv_heads;
  a.head_dim = c->head_dim;
  a.e2m1 = c->fmt == MX_E2M1 ? 1 : 0;
  a.block_table = block_table;
  a.kv_lens = kv_lens;
  a.q_starts = q_starts;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.T = T;
  a.status = static_cast<int*>(ws);
  return a;
}

}  // namespace mxk
