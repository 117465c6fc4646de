// C ABI of the operators that close a decoding step (MX projections, rotary positions,
// sandwich norms, sampling): argument checks and workspace carving (see include/mxmoe.h).
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/mxmoe.h"
#include "checks.h"
#include "internal.h"

using namespace mxk;

namespace {

// sizes whose products and grids fit their types
int check_linear(int T, int N, int K, int act_fmt, int w_fmt) {
  if (T < 0 || N <= 0 || K <= 0) return MX_ERR_INVALID_ARG;
  if ((act_fmt != MX_E4M3 && act_fmt != MX_E2M1) || (w_fmt != MX_E4M3 && w_fmt != MX_E2M1)) return MX_ERR_INVALID_ARG;
  if (K % 32 || K > (1 << 20) || N > (1 << 22) || T > (1 << 22) || (act_fmt == MX_E2M1 && w_fmt != MX_E2M1)) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

// Workspace of mx_linear: the status word, the tokens' tiled scales, their codes.
// (tokens' scales have as many blocks along K as the weights', an even number with E2M1)
size_t linear_scales_bytes(int T, int K) { return static_cast<size_t>((T + 127) / 128) * ((K + 255) / 256 * 2) * 512; }

}  // namespace

extern "C" {

size_t mx_linear_prepared_bytes(int N, int K, int fmt) {
  return check_linear(0, N, K, MX_E4M3, fmt) == MX_OK ? linear_layout(N, K, fmt).total_bytes : 0;
}

int mx_linear_prepare(const uint8_t* codes, const uint8_t* scales, int N, int K, int fmt, void* dst, size_t dst_bytes,
                      mx_stream_t stream) {
  const int st = check_linear(0, N, K, MX_E4M3, fmt);
  if (st != MX_OK) return st;
  if (!codes || !scales || !dst) return MX_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(dst, 256)) return MX_ERR_ALIGNMENT;
  const LinearLayout L = linear_layout(N, K, fmt);
  if (dst_bytes < L.total_bytes) return MX_ERR_WORKSPACE;
  return cuda_status(launch_linear_prepare(codes, scales, L, static_cast<uint8_t*>(dst), reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx_linear_workspace_size(int T, int N, int K, int act_fmt) {
  if (check_linear(T, N, K, act_fmt, MX_E2M1) != MX_OK) return 0;
  return 256 + al256(linear_scales_bytes(T, K)) + al256(static_cast<size_t>(T) * (act_fmt == MX_E2M1 ? K / 2 : K));
}

int mx_linear(const void* x_bf16, const uint8_t* codes, const uint8_t* scales, int act_fmt, const void* w_prep, int w_fmt,
              const float* bias, int T, int N, int K, void* out, int out_type, void* ws, size_t ws_bytes,
              mx_stream_t stream) {
  const int st = check_linear(T, N, K, act_fmt, w_fmt);
  if (st != MX_OK) return st;
  if (!type_ok(out_type)) return MX_ERR_INVALID_ARG;
  if (T == 0) return MX_OK;
  if (!w_prep || !out || !ws || !codes != !scales || !x_bf16 != (codes != nullptr)) return MX_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(w_prep, 256) || !aligned(bias, 4) || !aligned(out, 16) || !aligned(ws, 256))
    return MX_ERR_ALIGNMENT;
  if (ws_bytes < mx_linear_workspace_size(T, N, K, act_fmt)) return MX_ERR_WORKSPACE;
  uint8_t* const w = static_cast<uint8_t*>(ws);
  LinearArgs a{};
  a.w_prep = static_cast<const uint8_t*>(w_prep);
  a.w_fmt = w_fmt;
  a.act_fmt = act_fmt;
  a.x = x_bf16;
  a.scales = scales;
  a.t_scales = w + 256;
  a.t_codes = codes ? codes : w + 256 + al256(linear_scales_bytes(T, K));
  a.bias = bias;
  a.out = out;
  a.out_f32 = out_type == MX_F32;
  a.T = T;
  a.N = N;
  a.K = K;
  a.status = static_cast<int*>(ws);
  a.wait_limit_ns = wait_limit_ns();
  return cuda_status(launch_linear(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mx_sandwich_rmsnorm(const void* x, int x_type, const void* post_weight, int post_weight_type, const void* gate,
                        int gate_type, int gate_kind, int gate_act, const void* residual, int residual_type,
                        float residual_scale, float block_scale, const void* weight, int weight_type, int T, int H,
                        float eps, void* residual_out, void* y, int fmt, uint8_t* codes, uint8_t* scales,
                        mx_stream_t stream) {
  if (T < 0 || H <= 0 || !type_ok(x_type) || !type_ok(residual_type) || (post_weight && !type_ok(post_weight_type)) ||
      (weight && !type_ok(weight_type)) || !finite_positive(eps) || !std::isfinite(residual_scale) ||
      !std::isfinite(block_scale))
    return MX_ERR_INVALID_ARG;
  if (gate_kind < MX_GATE_NONE || gate_kind > MX_GATE_FULL || (gate_act != MX_GATE_ACT_NONE && gate_act != MX_GATE_ACT_SIGMOID) ||
      (gate_kind != MX_GATE_NONE && !type_ok(gate_type)))
    return MX_ERR_INVALID_ARG;
  if (codes && fmt != MX_E4M3 && fmt != MX_E2M1) return MX_ERR_INVALID_ARG;
  if (T == 0) return MX_OK;
  if (!x || !residual || !residual_out || !gate != (gate_kind == MX_GATE_NONE) || !codes != !scales) return MX_ERR_INVALID_ARG;
  if (weight ? !y && !codes : y || codes) return MX_ERR_INVALID_ARG;
  if (H % 32 || H > 32768) return MX_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(post_weight, 16) ||
      !aligned(weight, 16) || !aligned(y, 16) || !aligned(codes, 16))
    return MX_ERR_ALIGNMENT;
  if (!aligned(gate, gate_kind == MX_GATE_TOKEN ? gate_type == MX_F32 ? 4 : 2 : 16)) return MX_ERR_ALIGNMENT;
  SandwichArgs a{};
  a.x = x;
  a.post_weight = post_weight;
  a.gate = gate;
  a.residual = residual;
  a.weight = weight;
  a.x_f32 = x_type == MX_F32;
  a.post_weight_f32 = post_weight_type == MX_F32;
  a.gate_f32 = gate_type == MX_F32;
  a.residual_f32 = residual_type == MX_F32;
  a.weight_f32 = weight_type == MX_F32;
  a.gate_kind = gate_kind;
  a.gate_act = gate_act;
  a.residual_scale = residual_scale;
  a.block_scale = block_scale;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.residual_out = residual_out;
  a.y = y;
  a.e2m1 = fmt == MX_E2M1 ? 1 : 0;
  a.codes = codes;
  a.scales = scales;
  return cuda_status(launch_sandwich_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mx_rope_table(int rot_dim, double base, int scaling, double factor, double low, double high, int original_length,
                  uint64_t* turns, float* amplitude) {
  if (!turns || !amplitude || rot_dim <= 0 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base)) return MX_ERR_INVALID_ARG;
  if (scaling < MX_ROPE_SCALING_NONE || scaling > MX_ROPE_SCALING_BANDS) return MX_ERR_INVALID_ARG;
  if (scaling != MX_ROPE_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return MX_ERR_INVALID_ARG;
  const bool ramp = scaling == MX_ROPE_SCALING_YARN || scaling == MX_ROPE_SCALING_BANDS;
  if (ramp && (original_length <= 0 || !(low > 0.0) || !(high > low) || !std::isfinite(high))) return MX_ERR_INVALID_ARG;
  if (scaling == MX_ROPE_SCALING_NTK) {
    if (rot_dim == 2) return MX_ERR_INVALID_ARG;
    base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  }
  constexpr double kTwoPi = 6.283185307179586476925;
  *amplitude = scaling == MX_ROPE_SCALING_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  auto pair_of = [&](double t) { return rot_dim * std::log(original_length / (t * kTwoPi)) / (2.0 * std::log(base)); };
  const double from = ramp ? std::max(std::floor(pair_of(high)), 0.0) : 0.0;
  const double to = ramp ? std::min(std::ceil(pair_of(low)), rot_dim - 1.0) : 0.0;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    double slow = 0.0;  // the share of f / factor
    if (scaling == MX_ROPE_SCALING_LINEAR) slow = 1.0;
    else if (scaling == MX_ROPE_SCALING_YARN) slow = (i - from) / std::max(to - from, 0.001);
    else if (scaling == MX_ROPE_SCALING_BANDS) slow = 1.0 - (original_length * f / kTwoPi - low) / (high - low);
    slow = std::min(std::max(slow, 0.0), 1.0);
    if (slow > 0.0) f = f / factor * slow + f * (1.0 - slow);
    const double turn = f / kTwoPi;
    // below 2^64 for any fraction of a turn, whole turns do not count
    turns[i] = static_cast<uint64_t>(std::ldexp(turn - std::floor(turn), 64));
  }
  return MX_OK;
}

int mx_rope_kv_append(const mx_kv_cache* cache, const void* q, int64_t q_stride, int n_q_heads, void* q_out,
                      int64_t q_out_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      const int32_t* positions, const uint64_t* turns, int rot_dim, int layout, float amplitude,
                      const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts, int n_seqs,
                      int max_pages, int T, void* ws, size_t ws_bytes, mx_stream_t stream) {
  int st = check_cache(cache, n_seqs, max_pages, T);
  if (st != MX_OK) return st;
  const int64_t row = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
  if (k_stride < row || v_stride < row || n_q_heads < 0) return MX_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(n_q_heads) * cache->head_dim;
  if (n_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row)) return MX_ERR_INVALID_ARG;
  if ((layout != MX_ROPE_HALF && layout != MX_ROPE_INTERLEAVED) || rot_dim < 0 || rot_dim > cache->head_dim ||
      !std::isfinite(amplitude))
    return MX_ERR_INVALID_ARG;
  if (rot_dim % 16 || cache->head_dim > 256 || q_row > (1 << 20)) return MX_ERR_UNSUPPORTED;
  if (T == 0 || n_seqs == 0) return MX_OK;
  if (!k || !v || !q != (n_q_heads == 0) || !q != !q_out || (rot_dim > 0 && !turns)) return MX_ERR_INVALID_ARG;
  st = check_cache_pointers(cache, block_table, kv_lens, q_starts, ws, ws_bytes);
  if (st != MX_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 || v_stride % 8 || !aligned(positions, 4) || !aligned(turns, 8))
    return MX_ERR_ALIGNMENT;
  if (n_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 || q_out_stride % 8)) return MX_ERR_ALIGNMENT;
  RopeArgs r{};
  r.kv = kv_args(cache, block_table, kv_lens, q_starts, n_seqs, max_pages, T, ws);
  r.kv.k = k;
  r.kv.v = v;
  r.kv.k_stride = k_stride;
  r.kv.v_stride = v_stride;
  r.q = q;
  r.q_out = q_out;
  r.q_stride = q_stride;
  r.q_out_stride = q_out_stride;
  r.n_q_heads = n_q_heads;
  r.positions = positions;
  r.turns = turns;
  r.rot = rot_dim;
  r.interleaved = layout == MX_ROPE_INTERLEAVED;
  r.amplitude = amplitude;
  return cuda_status(launch_rope_kv_append(r, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx_sample_workspace_size(int T, int V) { return T < 0 || V <= 0 ? 0 : 256; }

int mx_sample(const void* logits, int type, int64_t stride, int T, int V, const float* temperature, const int32_t* top_k,
              const float* top_p, const float* min_p, const float* u, int32_t* tokens, float* logp, void* ws,
              size_t ws_bytes, mx_stream_t stream) {
  if (T < 0 || V <= 0 || !type_ok(type) || stride < V) return MX_ERR_INVALID_ARG;
  if (!sample_supported(V, type == MX_BF16) || T > INT_MAX / 16) return MX_ERR_UNSUPPORTED;
  if (T == 0) return MX_OK;
  if (!logits || !u || !tokens || !ws) return MX_ERR_INVALID_ARG;
  if (!aligned(logits, type == MX_BF16 ? 2 : 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(ws, 256))
    return MX_ERR_ALIGNMENT;
  if (ws_bytes < mx_sample_workspace_size(T, V)) return MX_ERR_WORKSPACE;
  SampleArgs a{};
  a.logits = logits;
  a.stride = stride;
  a.bf16 = type == MX_BF16;
  a.T = T;
  a.V = V;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.tokens = tokens;
  a.logp = logp;
  a.status = static_cast<int*>(ws);
  return cuda_status(launch_sample(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
