"""One decoder block around the expert layer, as a serving loop runs it:

    norm -> q, k, v -> into the paged MX cache -> attention over it -> projection
    -> norm, whose MX codes are the experts' activations -> router -> experts

The dense projections are plain matrix products; everything else is a call of
this library on the current stream, without a host synchronisation.  The batch is
ragged: prompts, chunks of prompts and single new tokens go through one call.

``python -m block_scaled_mx_gb300.block`` serves a few sequences of random
tokens through two blocks: a prompt step, then single-token steps.
"""
import torch

from . import mxmoe as mx


class DecoderBlock:
    """Weights (bf16): ``w_qkv`` [(n_heads + 2 n_kv_heads) head_dim, H], ``w_o``
    [H, n_heads head_dim], the norms' ``g_attn`` and ``g_mlp`` [H], ``w_router``
    [E, H]; ``experts`` is a prepared MoELayer.

    Calls on different streams may overlap: each stream has workspaces of its own,
    which the block keeps (at most 41 MB for the attention, and what the experts'
    GEMMs need).  An object is for one host thread at a time.

    With ``keep_last`` the block holds what its last call computed on the way in
    ``last`` (q and with it the whole projection, att, y, codes, scales) until the
    next call."""

    def __init__(self, w_qkv, w_o, g_attn, g_mlp, w_router, experts, n_heads, n_kv_heads, head_dim, eps=1e-6, window=0,
                 keep_last=False):
        self.w_qkv, self.w_o, self.g_attn, self.g_mlp, self.w_router, self.experts = w_qkv, w_o, g_attn, g_mlp, w_router, experts
        self.n_heads, self.n_kv_heads, self.head_dim, self.eps, self.window = n_heads, n_kv_heads, head_dim, eps, window
        self.keep_last, self.last = keep_last, None
        self._ws = {}  # by name and stream

    def _workspace(self, name, nbytes):
        key = name, mx.current_stream()
        ws = self._ws.get(key)
        if ws is None or ws.nbytes < nbytes:
            old, ws = ws, mx.alloc_workspace(nbytes)
            if old is not None:
                ws[:4] = old[:4]  # an error that status() has not read yet
            self._ws[key] = ws
        return ws

    def forward(self, x, residual, cache, block_table, kv_lens, q_starts, max_q_len):
        """x [T, H] (bf16, or the fp32 output of the block before) and the residual
        stream (bf16) -> the experts' output [T, H] fp32 and the new residual stream.
        ``kv_lens`` counts the new tokens; ``q_starts`` says whose they are."""
        T, H = x.shape
        dev = x.device
        e, hq, hk, d = self.experts, self.n_heads, self.n_kv_heads, self.head_dim
        batch = (block_table, kv_lens, q_starts)
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)

        if T == 0:  # no sequence has a new token
            return torch.empty(0, H, dtype=torch.float32, device=dev), torch.empty(0, H, **bf16)
        y, mid, after = torch.empty(T, H, **bf16), torch.empty(T, H, **bf16), torch.empty(T, H, **bf16)
        mx.mx_add_rmsnorm(x, self.g_attn, self.eps, residual=residual, residual_out=mid, y=y)
        qkv = (y @ self.w_qkv.t()).view(T, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]   # read where they lie
        need = mx.mx_paged_attention_workspace_size(T, kv_lens.numel(), hq, hk, d, max_q_len)
        ws = self._workspace("attention", need)
        mx.mx_kv_append(cache, k, v, *batch, ws)
        att = torch.empty(T, hq, d, **bf16)
        mx.mx_paged_attention(q, cache, *batch, att, ws, window=self.window, max_q_len=max_q_len)

        codes = torch.empty(T, H, dtype=torch.uint8, device=dev)
        scales = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
        mx.mx_add_rmsnorm(att.view(T, hq * d) @ self.w_o.t(), self.g_mlp, self.eps, residual=mid, residual_out=after, y=y,
                          codes=codes, scales=scales)
        ids, weights = torch.empty(T, e.k, **i32), torch.empty(T, e.k, dtype=torch.float32, device=dev)
        mx.moe_route_gemm_topk(y, self.w_router, e.k, self._workspace("router", 256 + 4 * 128 * e.E), topk_ids=ids,
                               topk_w=weights)
        slots = T * (e.k + 1)
        counts, offsets, order = (torch.empty(n, **i32) for n in (e.E + 1, e.E + 2, slots))
        mx.moe_permute(ids, e.E, counts, offsets, order,
                       self._workspace("permute", mx.moe_permute_workspace_size(T, e.E, e.k)))
        sizes = (e.fmt, T, H, e.I, e.E, e.k)
        h_codes = torch.empty(slots, e.I, dtype=torch.uint8, device=dev)
        h_scales = torch.empty(slots, e.I // 32, dtype=torch.uint8, device=dev)
        ws = self._workspace("experts", mx.moe_gemm_workspace_size(T, H, e.I, e.E, e.k))
        mx.moe_grouped_gemm_swiglu(codes, scales, offsets, order, e.w1, *sizes, h_codes, h_scales, ws)
        out = torch.zeros(T, H, dtype=torch.float32, device=dev)
        mx.moe_grouped_gemm_down_combine(h_codes, h_scales, offsets, order, weights, e.w2, *sizes, out, ws)
        if self.keep_last:
            self.last = dict(q=q, att=att, y=y, codes=codes, scales=scales)
        return out, after

    def status(self):
        """The first error that a kernel reported (waits for the device), 0 for none."""
        torch.cuda.synchronize()
        return max((mx.moe_get_status(ws, stream) for (_, stream), ws in self._ws.items()), default=0)


def random_block(H, I, E, k, n_heads, n_kv_heads, head_dim, fmt="e4m3", window=0, seed=0, device="cuda", keep_last=True):
    """A block of random weights, which keeps what its last call computed unless told
    not to."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, fan_in):
        return torch.randn(*shape, generator=g, device=device) * fan_in ** -0.5

    half = 2 if mx.FORMATS[fmt] == mx.MX_E2M1 else 1
    tables = []
    for rows, cols in ((2 * I, H), (H, I)):
        codes = torch.empty(E + 1, rows, cols // half, dtype=torch.uint8, device=device)
        scales = torch.empty(E + 1, rows, cols // 32, dtype=torch.uint8, device=device)
        for i in range(E + 1):
            mx.mx_quantize_weights(normal(rows, cols, fan_in=cols), mx.FORMATS[fmt], codes[i], scales[i])
        tables += [codes, scales]
    experts = mx.MoELayer(*tables, mx.FORMATS[fmt], H, I, E, k)
    bf16 = torch.bfloat16
    return DecoderBlock(normal((n_heads + 2 * n_kv_heads) * head_dim, H, fan_in=H).to(bf16),
                        normal(H, n_heads * head_dim, fan_in=n_heads * head_dim).to(bf16),
                        torch.ones(H, dtype=bf16, device=device), torch.ones(H, dtype=bf16, device=device),
                        normal(E, H, fan_in=H).to(bf16), experts, n_heads, n_kv_heads, head_dim, window=window,
                        keep_last=keep_last)


def main(prompts=(700, 33, 1), steps=4, H=2048, I=512, E=16, k=4, n_heads=16, n_kv_heads=2, head_dim=128, page=64):
    blocks = [random_block(H, I, E, k, n_heads, n_kv_heads, head_dim, seed=s, keep_last=False) for s in range(2)]
    n = len(prompts)
    per = -(-(max(prompts) + steps) // page)
    table = torch.randperm(n * per, device="cuda").to(torch.int32).view(n, per)
    caches = [mx.KVCache(n * per, page, n_kv_heads, head_dim) for _ in blocks]
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    for step in range(steps + 1):
        new = list(prompts) if step == 0 else [1] * n
        starts = torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        x = torch.randn(sum(new), H, device="cuda").to(torch.bfloat16)
        residual = torch.zeros_like(x)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for block, cache in zip(blocks, caches):
            x, residual = block.forward(x, residual, cache, table, lens, starts, max(new))
        end.record()
        status = max(block.status() for block in blocks)
        if status:
            raise mx.MxError(status, "decoder block")
        print(f"step {step}: {sum(new)} new tokens, caches of {lens.tolist()}, {begin.elapsed_time(end):.3f} ms, "
              f"|out| {float(x.abs().mean()):.4f}")


if __name__ == "__main__":
    main()
