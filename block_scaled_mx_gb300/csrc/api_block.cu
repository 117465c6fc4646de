// C ABI of the operators around the expert layer (residual norm, paged MX cache,
// attention): argument checks and workspace carving (see include/mxmoe.h).
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/mxmoe.h"
#include "internal.h"

using namespace mxk;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }
bool type_ok(int t) { return t == MX_BF16 || t == MX_F32; }
bool finite_positive(float v) { return v > 0.0f && v <= 3.402823466e38f; }

// The cache and the batch's sizes, as all three cache calls take them.
int check_cache(const mx_kv_cache* c, int n_seqs, int max_pages, int T) {
  if (!c || T < 0 || n_seqs < 0 || max_pages <= 0) return MX_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0) return MX_ERR_INVALID_ARG;
  if (c->fmt != MX_E4M3 && c->fmt != MX_E2M1) return MX_ERR_INVALID_ARG;
  if (c->head_dim % 32) return MX_ERR_UNSUPPORTED;
  // positions, heads x elements and grid sizes are ints
  if (static_cast<int64_t>(max_pages) * c->page_size > INT_MAX / 2) return MX_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->n_kv_heads) * c->head_dim > (1 << 20) || T > INT_MAX / 2) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

int check_cache_pointers(const mx_kv_cache* c, const void* block_table, const void* kv_lens, const void* q_starts,
                         const void* ws, size_t ws_bytes) {
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !block_table || !kv_lens || !q_starts || !ws)
    return MX_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16) ||
      !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_starts, 4) || !aligned(ws, 256))
    return MX_ERR_ALIGNMENT;
  return ws_bytes < 256 ? MX_ERR_WORKSPACE : MX_OK;
}

KvArgs kv_args(const mx_kv_cache* c, const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts,
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

// Attention workspace: the status word, the segments' arrival counters, then
// the split segments' partial results.
constexpr size_t kArrivedOffset = 256;
constexpr size_t kArrivedBytes = sizeof(unsigned) * kAttnMaxCtas;

// Which kernel takes which sequences: all go to the few-rows kernel, all to the chunk
// kernel, or those of up to `split` rows (new tokens x query heads of a KV head) to the
// one and the others to the other, in two launches.
//
// The few-rows kernel goes through the keys again for every 8 rows; the chunk kernel
// takes as long for 256 as for one, but starts and ends slower, the more so the fewer
// the (sequence, KV head) pairs among which its 152 CTAs share out and join the keys.
// Count a batch's work in 64-key units, and 8 more for each pair.  Without the start the
// chunk kernel's time is that of two or three tiles of 8 rows; every further tile costs
// the few-rows kernel 2.5 ns a unit (heads of 128 in MXFP8; 1.6 to 2.8 in the other
// three forms), and the start is worth 10 us and 200 us over the number of pairs, less
// where a pair has few units.  Two launches start and end twice; they pay where many
// pairs have one tile, by which the few-rows kernel is ahead as a chunk's segment costs
// 16 units beside its keys.
// In us, few rows / chunk, heads of 128 in MXFP8, equal sequences:
//   pairs x keys     rows and times
//   2 x 2048         128: 23 / 40
//   2 x 131072       64: 102 / 167     96: 140 / 169     128: 180 / 170
//   16 x 2048        96: 35 / 41       128: 42 / 41
//   16 x 8192        32: 36 / 47       48: 47 / 47       64: 57 / 47
//   16 x 131072      16: 182 / 191     24: 255 / 192     128: 1293 / 204
//   32 x 2048        48: 32 / 39       64: 39 / 39       96: 52 / 41
//   64 x 8192        16: 59 / 69       24: 80 / 71
// and few rows / chunk / two launches, lengths of a quarter to all of the keys:
//   16 x 32768, 3 to 6 tokens of 8 rows         75 / 82 / 118
//   64 x 8192, one of 6 tokens, others of one    33 / 62 / 75
//   16 x 2048, one of 512 tokens, others of one  - / 45 / 59
//   512 x 2048, the same                         - / 146 / 91
//   192 x 5000, heads of 64, window of 2048,
//     12 of 24 sequences of 139 to 700 tokens    - / 274 / 272
// Over 1326 batches (1 to 512 pairs, 512 to 131072 keys, both head sizes and formats) the
// rule takes 0.3% longer than the fastest of the three, and 38% at worst.
//
// The lengths are on the device.  Keys are counted by what bounds them, the block
// table's width and the window; rows by the average over the sequences; and for two
// launches the batch is taken to be of single tokens and of as many of max_q_len as T
// has room for.
constexpr int kMostFewRows = 128;
struct AttnChoice {
  bool few;   // all to the few-rows kernel
  int split;  // else those of up to this many rows
};
AttnChoice choose_kernel(int T, int n_seqs, int n_kv_heads, int group, int max_q_len, int head_dim, bool e2m1, int64_t keys) {
  const int even = head_dim == 128 && !e2m1 ? 2 : 3;
  const double pairs = static_cast<double>(n_seqs) * n_kv_heads, units = static_cast<double>((keys + 63) / 64);
  const int64_t most = static_cast<int64_t>(max_q_len) * group;
  if (most <= kMostFewRows) {
    const double tiles = std::min(static_cast<double>((most + 7) / 8), static_cast<double>(T) * group / n_seqs / 8);
    const double start = std::min(260 * units, 4000 + 80000 / pairs);  // of the chunk kernel, in units of one tile
    if (tiles <= even || (tiles - even) * pairs * (units + 8) <= start) return {true, 0};
  }
  if (T >= static_cast<int64_t>(n_seqs) * max_q_len) return {false, 0};  // room for max_q_len in all of them
  const double single = n_seqs - static_cast<double>(T - n_seqs) / std::max(max_q_len - 1, 1);
  const bool pays = single * n_kv_heads * ((units + 16) * even - (units + 8)) > 16000;  // ahead by a second start
  return {false, pays ? 8 * (even - 1) : 0};
}

int check_attention(int T, int n_seqs, int n_heads, int n_kv_heads, int head_dim, int max_q_len) {
  if (T < 0 || n_seqs < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || max_q_len < 0) return MX_ERR_INVALID_ARG;
  if (n_heads % n_kv_heads) return MX_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MX_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(T) * n_heads > (1 << 30) || n_heads > (1 << 14)) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

}  // namespace

extern "C" {

int mx_add_rmsnorm(const void* x, int x_type, const void* residual, int residual_type, const void* weight,
                   int weight_type, int T, int H, float eps, void* residual_out, void* y, int fmt, uint8_t* codes,
                   uint8_t* scales, mx_stream_t stream) {
  if (T < 0 || H <= 0 || !type_ok(x_type) || !type_ok(weight_type) || (residual && !type_ok(residual_type)) ||
      !finite_positive(eps))
    return MX_ERR_INVALID_ARG;
  if (codes && fmt != MX_E4M3 && fmt != MX_E2M1) return MX_ERR_INVALID_ARG;
  if (T == 0) return MX_OK;
  if (!x || !weight || (!y && !codes) || !codes != !scales || !residual != !residual_out) return MX_ERR_INVALID_ARG;
  if (H % 32 || H > 32768) return MX_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(codes, 16))
    return MX_ERR_ALIGNMENT;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.x_f32 = x_type == MX_F32;
  a.residual_f32 = residual_type == MX_F32;
  a.weight_f32 = weight_type == MX_F32;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.residual_out = residual_out;
  a.y = y;
  a.e2m1 = fmt == MX_E2M1 ? 1 : 0;
  a.codes = codes;
  a.scales = scales;
  return cuda_status(launch_add_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mx_kv_append(const mx_kv_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts, int n_seqs,
                 int max_pages, int T, void* ws, size_t ws_bytes, mx_stream_t stream) {
  int st = check_cache(cache, n_seqs, max_pages, T);
  if (st != MX_OK) return st;
  const int64_t row = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
  if (k_stride < row || v_stride < row) return MX_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return MX_OK;
  if (!k || !v) return MX_ERR_INVALID_ARG;
  st = check_cache_pointers(cache, block_table, kv_lens, q_starts, ws, ws_bytes);
  if (st != MX_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8) return MX_ERR_ALIGNMENT;
  KvArgs a = kv_args(cache, block_table, kv_lens, q_starts, n_seqs, max_pages, T, ws);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  return cuda_status(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mx_kv_read(const mx_kv_cache* cache, const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts,
               int n_seqs, int max_pages, int T, void* k_out, void* v_out, void* ws, size_t ws_bytes,
               mx_stream_t stream) {
  int st = check_cache(cache, n_seqs, max_pages, T);
  if (st != MX_OK) return st;
  if (T == 0) return MX_OK;
  if (!k_out || !v_out) return MX_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return MX_ERR_ALIGNMENT;
  if (n_seqs == 0) {  // all rows are padding
    const size_t bytes = static_cast<size_t>(T) * cache->n_kv_heads * cache->head_dim * 2;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cudaMemsetAsync(k_out, 0, bytes, s) == cudaSuccess ? cuda_status(cudaMemsetAsync(v_out, 0, bytes, s)) : MX_ERR_CUDA;
  }
  st = check_cache_pointers(cache, block_table, kv_lens, q_starts, ws, ws_bytes);
  if (st != MX_OK) return st;
  KvArgs a = kv_args(cache, block_table, kv_lens, q_starts, n_seqs, max_pages, T, ws);
  a.k_out = k_out;
  a.v_out = v_out;
  return cuda_status(launch_kv_read(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx_paged_attention_workspace_size(int T, int n_seqs, int n_heads, int n_kv_heads, int head_dim, int max_q_len) {
  if (check_attention(T, n_seqs, n_heads, n_kv_heads, head_dim, max_q_len) != MX_OK) return 0;
  size_t part = attn_rows_part_bytes(head_dim);
  // up to 16 rows are the few-rows kernel's whatever the lengths, which are not known here
  if (static_cast<int64_t>(max_q_len) * (n_heads / n_kv_heads) > 16) part = std::max(part, attn_chunk_part_bytes(head_dim));
  return kArrivedOffset + al256(kArrivedBytes) + part;
}

int mx_paged_attention(const mx_kv_cache* cache, const void* q, int64_t q_stride, int n_heads,
                       const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts, int n_seqs,
                       int max_pages, int T, int max_q_len, float scale, int causal, int window, void* out, float* lse,
                       void* ws, size_t ws_bytes, mx_stream_t stream) {
  int st = check_cache(cache, n_seqs, max_pages, T);
  if (st != MX_OK) return st;
  st = check_attention(T, n_seqs, n_heads, cache->n_kv_heads, cache->head_dim, max_q_len);
  if (st != MX_OK) return st;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!finite_positive(scale) || !finite_positive(scale_log2) || window < 0 || (window > 0 && !causal)) return MX_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(n_heads) * cache->head_dim) return MX_ERR_INVALID_ARG;
  if (cache->page_size % 16) return MX_ERR_UNSUPPORTED;
  // cache rows are counted in ints
  if (static_cast<int64_t>(cache->num_pages) * cache->page_size > INT_MAX / cache->n_kv_heads) return MX_ERR_UNSUPPORTED;
  // Places of work are counted in 32 bits, those of one KV head in a signed int.  At
  // most: 256-row tiles, and 8-row ones of the sequences with few rows, times 64-key
  // units and a tile's cost.
  const double tiles = static_cast<double>(T) * (n_heads / cache->n_kv_heads) / 256 + n_seqs * (1.0 + kMostFewRows / 8);
  const double places = tiles * (static_cast<double>(max_pages) * cache->page_size / 64 + 32);
  if (places > 2147483647.0 || places * cache->n_kv_heads > 4.0e9) return MX_ERR_UNSUPPORTED;
  if (T == 0 || n_seqs == 0 || max_q_len == 0) return MX_OK;
  if (!q || !out) return MX_ERR_INVALID_ARG;
  st = check_cache_pointers(cache, block_table, kv_lens, q_starts, ws, ws_bytes);
  if (st != MX_OK) return st;
  if (!aligned(q, 16) || q_stride % 8 || !aligned(out, 16) || !aligned(lse, 4)) return MX_ERR_ALIGNMENT;
  if (ws_bytes < mx_paged_attention_workspace_size(T, n_seqs, n_heads, cache->n_kv_heads, cache->head_dim, max_q_len))
    return MX_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k_codes = cache->k_codes;
  a.k_scales = cache->k_scales;
  a.v_codes = cache->v_codes;
  a.v_scales = cache->v_scales;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.e2m1 = cache->fmt == MX_E2M1 ? 1 : 0;
  a.block_table = block_table;
  a.kv_lens = kv_lens;
  a.q_starts = q_starts;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.T = T;
  a.group = n_heads / cache->n_kv_heads;
  a.group_div = FastDiv::by(a.group);
  a.page_div = FastDiv::by(a.page_size);
  a.max_q_len = max_q_len;
  a.causal = causal != 0;
  a.window = window;
  a.scale_log2 = scale_log2;
  a.out = out;
  a.lse = lse;
  a.status = static_cast<int*>(ws);
  a.arrived = reinterpret_cast<unsigned*>(w + kArrivedOffset);
  a.part_ml = reinterpret_cast<float2*>(w + kArrivedOffset + al256(kArrivedBytes));
  a.wait_limit_ns = wait_limit_ns();
  a.box_keys = a.page_size % 64 == 0 ? 64 : a.page_size % 32 == 0 ? 32 : 16;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  a.rows_above = 0;
  a.rows_upto = INT_MAX;
  int64_t keys = static_cast<int64_t>(max_pages) * a.page_size;
  if (window > 0) keys = std::min(keys, static_cast<int64_t>(window) + max_q_len);
  const AttnChoice choice = choose_kernel(T, n_seqs, a.n_kv_heads, a.group, max_q_len, a.head_dim, a.e2m1 != 0, keys);
  if (choice.few) return cuda_status(launch_attn_rows(a, cs));
  if (choice.split > 0) {
    a.rows_upto = choice.split;
    st = cuda_status(launch_attn_rows(a, cs));
    if (st != MX_OK) return st;
    a.rows_above = choice.split;
    a.rows_upto = INT_MAX;
  }
  return cuda_status(launch_attn_chunk(a, cs));
}

}  // extern "C"
