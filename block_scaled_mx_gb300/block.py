"""One decoder block around the expert layer, as a serving loop runs it, and what turns
its output into tokens:

    norm -> q, k, v -> positions, and into the paged MX cache -> attention over it
    -> projection -> norm, whose MX codes are the experts' activations -> router -> experts
    ... -> norm -> logits -> a token for each sequence

The dense projections are plain matrix products or, with MX weights, this library's;
everything else is a call of this library on the current stream, without a host
synchronisation.  The batch is ragged: prompts, chunks of prompts and single new tokens
go through one call.

``python -m block_scaled_mx_gb300.block`` generates tokens for a few prompts with two
blocks of random weights: a prompt step, then single-token steps.
"""
import torch

from . import mxmoe as mx


class Sandwich:
    """What happens to a sub-block's output x on its way into the residual stream
    (mx_sandwich_rmsnorm): z = residual_scale * residual + block_scale * act(gate) * n, with
    n = RMSNorm(x) * post, or x where there is no ``post`` weight [H]; ``gate`` [H] or None."""

    def __init__(self, post=None, gate=None, gate_act="none", block_scale=1.0, residual_scale=1.0):
        self.post, self.gate, self.gate_act, self.block_scale, self.residual_scale = post, gate, gate_act, block_scale, residual_scale


def _norm(sandwich, x, weight, eps, residual, residual_out, **out):
    """The norm ahead of a sub-block, with the residual and a Sandwich or without one."""
    if sandwich is None:
        mx.mx_add_rmsnorm(x, weight, eps, residual=residual, residual_out=residual_out, **out)
    else:
        mx.mx_sandwich_rmsnorm(x, sandwich.post, eps, residual, residual_out, gate=sandwich.gate, gate_act=sandwich.gate_act,
                               block_scale=sandwich.block_scale, residual_scale=sandwich.residual_scale, weight=weight, **out)


class _Workspaces:
    """Workspaces by name and stream, which are kept: calls on different streams may overlap.
    So may the graphs that calls are captured into: each has workspaces of its own, which
    are kept as long as the object."""

    def __init__(self):
        self._ws = {}        # by name, stream and capture
        self._outgrown = []  # workspaces that earlier calls of a capture go on using, with their stream

    def _workspace(self, name, nbytes):
        key = name, mx.current_stream(), mx.current_capture()
        ws = self._ws.get(key)
        if ws is None or ws.nbytes < nbytes:
            old = ws
            if key[2]:
                ws = mx.alloc_captured_workspace(nbytes)
                if old is not None:
                    self._outgrown.append((key[1], old))
            else:
                ws = mx.alloc_workspace(nbytes)
                if old is not None:
                    ws[:4] = old[:4]  # an error that status() has not read yet
            self._ws[key] = ws
        return ws

    def _project(self, w, x=None, codes=None, scales=None, out_type=torch.bfloat16):
        """x (bf16), or its MX codes, times the transposed weights: bf16 [N, K] or LinearWeights."""
        if not isinstance(w, mx.LinearWeights):
            return x @ w.t()
        T = (codes if x is None else x).shape[0]
        out = torch.empty(T, w.N, dtype=out_type, device=w.data.device)
        ws = self._workspace("linear", mx.mx_linear_workspace_size(T, w.N, w.K))
        mx.mx_linear(w, out, ws, x=x, codes=codes, scales=scales)
        return out

    def status(self):
        """The first error that a kernel reported (waits for the device), 0 for none."""
        torch.cuda.synchronize()
        every = [(stream, ws) for (_, stream, _), ws in self._ws.items()] + self._outgrown
        return max((mx.moe_get_status(ws, stream) for stream, ws in every), default=0)


class DecoderBlock(_Workspaces):
    """Weights: ``w_qkv`` [(n_heads + 2 n_kv_heads) head_dim, H] and ``w_o`` [H, n_heads
    head_dim], bf16 or MX (LinearWeights), the norms' ``g_attn`` and ``g_mlp`` [H] and
    ``w_router`` [E, H] in bf16; ``experts`` is a prepared MoELayer.  ``rope`` gives the
    queries and keys their positions; ``before`` and ``between`` are the Sandwich of the
    incoming x (the output of the block before) and of the attention's projection.

    Calls on different streams may overlap, and so may graphs that calls are captured into:
    each stream and each graph has workspaces of its own, which the block keeps (at most
    41 MB for the attention, and what the experts' GEMMs and the projections need).  An
    object is for one host thread at a time.

    With ``keep_last`` the block holds what its last call computed on the way in
    ``last`` (q and with it the whole projection, att, y, codes, scales) until the
    next call."""

    def __init__(self, w_qkv, w_o, g_attn, g_mlp, w_router, experts, n_heads, n_kv_heads, head_dim, eps=1e-6, window=0,
                 keep_last=False, rope=None, before=None, between=None):
        super().__init__()
        self.w_qkv, self.w_o, self.g_attn, self.g_mlp, self.w_router, self.experts = w_qkv, w_o, g_attn, g_mlp, w_router, experts
        self.n_heads, self.n_kv_heads, self.head_dim, self.eps, self.window = n_heads, n_kv_heads, head_dim, eps, window
        self.rope, self.before, self.between = rope, before, between
        self.keep_last, self.last = keep_last, None

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
        codes = torch.empty(T, H, dtype=torch.uint8, device=dev)
        scales = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
        if isinstance(self.w_qkv, mx.LinearWeights):  # the norm's codes are the projection's activations
            _norm(self.before, x, self.g_attn, self.eps, residual, mid, codes=codes, scales=scales)
            qkv = self._project(self.w_qkv, codes=codes, scales=scales)
        else:
            _norm(self.before, x, self.g_attn, self.eps, residual, mid, y=y)
            qkv = self._project(self.w_qkv, y)
        qkv = qkv.view(T, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]   # read where they lie
        need = mx.mx_paged_attention_workspace_size(T, kv_lens.numel(), hq, hk, d, max_q_len)
        ws = self._workspace("attention", need)
        if self.rope is None:
            mx.mx_kv_append(cache, k, v, *batch, ws)
        else:
            mx.mx_rope_kv_append(cache, self.rope, q, k, v, *batch, ws, q_out=q)   # q where it lies
        att = torch.empty(T, hq, d, **bf16)
        mx.mx_paged_attention(q, cache, *batch, att, ws, window=self.window, max_q_len=max_q_len)

        _norm(self.between, self._project(self.w_o, att.view(T, hq * d)), self.g_mlp, self.eps, mid, after, y=y, codes=codes,
              scales=scales)
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


class TokenHead(_Workspaces):
    """From the last block's output to tokens: the final norm ``g`` [H], logits through
    ``w`` [V, H] (bf16 or MX), and a draw by given random numbers.  ``before`` is the
    Sandwich of the incoming x."""

    def __init__(self, g, w, eps=1e-6, before=None):
        super().__init__()
        self.g, self.w, self.eps, self.before = g, w, eps, before

    def forward(self, x, residual, u, temperature=None, top_k=None, top_p=None, min_p=None):
        """x [n, H] (fp32 or bf16) and the residual stream (bf16): the rows that tokens are
        wanted for -> tokens int32 [n], their log-probabilities fp32 [n] and the logits."""
        n, H = x.shape
        dev = x.device
        rest = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
        if isinstance(self.w, mx.LinearWeights):
            codes = torch.empty(n, H, dtype=torch.uint8, device=dev)
            scales = torch.empty(n, H // 32, dtype=torch.uint8, device=dev)
            _norm(self.before, x, self.g, self.eps, residual, rest, codes=codes, scales=scales)
            logits = self._project(self.w, codes=codes, scales=scales, out_type=torch.float32)
        else:
            y = torch.empty(n, H, dtype=torch.bfloat16, device=dev)
            _norm(self.before, x, self.g, self.eps, residual, rest, y=y)
            logits = self._project(self.w, y)
        tokens = torch.empty(n, dtype=torch.int32, device=dev)
        logp = torch.empty(n, dtype=torch.float32, device=dev)
        ws = self._workspace("sample", mx.mx_sample_workspace_size(n, logits.shape[1]))
        mx.mx_sample(logits, u, tokens, ws, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, logp=logp)
        return tokens, logp, logits


def random_weights(w, fmt):
    """LinearWeights of an fp32 weight [N, K], quantised here."""
    N, K = w.shape
    codes = torch.empty(N, K // (2 if mx.FORMATS[fmt] == mx.MX_E2M1 else 1), dtype=torch.uint8, device=w.device)
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device=w.device)
    mx.mx_quantize_weights(w.contiguous(), fmt, codes, scales)
    return mx.LinearWeights(codes, scales, fmt)


def random_block(H, I, E, k, n_heads, n_kv_heads, head_dim, fmt="e4m3", window=0, seed=0, device="cuda", keep_last=True,
                 projections=None, **parts):
    """A block of random weights, which keeps what its last call computed unless told
    not to.  ``projections``: the format of MX projections (None: bf16); ``parts``: the
    block's rope, before and between."""
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

    def dense(w):
        return w.to(bf16) if projections is None else random_weights(w, projections)

    return DecoderBlock(dense(normal((n_heads + 2 * n_kv_heads) * head_dim, H, fan_in=H)),
                        dense(normal(H, n_heads * head_dim, fan_in=n_heads * head_dim)),
                        torch.ones(H, dtype=bf16, device=device), torch.ones(H, dtype=bf16, device=device),
                        normal(E, H, fan_in=H).to(bf16), experts, n_heads, n_kv_heads, head_dim, window=window,
                        keep_last=keep_last, **parts)


def main(prompts=(700, 33, 1), steps=4, H=2048, I=512, E=16, k=4, n_heads=16, n_kv_heads=2, head_dim=128, page=64, vocabulary=32003):
    bf16 = torch.bfloat16
    rope = mx.Rope(head_dim)
    ones = torch.ones(H, dtype=bf16, device="cuda")
    post = Sandwich(post=ones, block_scale=0.5)
    blocks = [random_block(H, I, E, k, n_heads, n_kv_heads, head_dim, seed=s, keep_last=False, projections="e2m1", rope=rope,
                           before=post if s else None, between=post) for s in range(2)]
    g = torch.Generator(device="cuda").manual_seed(9)
    embedding = torch.randn(vocabulary, H, generator=g, device="cuda").to(bf16)
    head = TokenHead(ones, random_weights(torch.randn(vocabulary, H, generator=g, device="cuda") * H ** -0.5, "e4m3"), before=post)
    n = len(prompts)
    per = -(-(max(prompts) + steps) // page)
    table = torch.randperm(n * per, device="cuda").to(torch.int32).view(n, per)
    caches = [mx.KVCache(n * per, page, n_kv_heads, head_dim) for _ in blocks]
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, vocabulary, (sum(prompts),), generator=g, device="cuda")
    rules = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"),
                 top_p=torch.full((n,), 0.95, device="cuda"))
    for step in range(steps + 1):
        new = list(prompts) if step == 0 else [1] * n
        starts = torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        u = torch.rand(n, generator=g, device="cuda")
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        x = embedding[tokens]
        residual = torch.zeros_like(x)
        for block, cache in zip(blocks, caches):
            x, residual = block.forward(x, residual, cache, table, lens, starts, max(new))
        last = (starts[1:] - 1).long()   # each sequence's last token
        tokens, logp, _ = head.forward(x[last], residual[last], u, **rules)
        end.record()
        status = max([block.status() for block in blocks] + [head.status()])
        if status:
            raise mx.MxError(status, "decoder block")
        print(f"step {step}: {sum(new)} new tokens, caches of {lens.tolist()}, {begin.elapsed_time(end):.3f} ms, "
              f"next {tokens.tolist()}, log p {[round(v, 2) for v in logp.tolist()]}")


if __name__ == "__main__":
    main()
