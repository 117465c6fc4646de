"""The serving operators around the expert layer, as cases that can be timed and compared.

Three operators, which a decoder block calls one after the other:

  norm     residual addition, root-mean-square norm and MX quantisation in one pass (``mx_add_rmsnorm``)
  append   quantising new keys and values into a paged MX cache as they are written (``mx_kv_append``)
  read     reading a stretch of that cache back as bf16 (``mx_kv_read``)
  attend   attention of a chunk of new tokens over the cache (``mx_paged_attention``)

``run`` computes a case either in plain torch operations (``own`` false) or through this package (``own`` true).
Codes come back as float8_e4m3fn and block scales as float8_e8m0fnu views, that is as the values they stand for.
"""
import math
import random

import torch

own = False

BLOCK = 32  # elements that share one E8M0 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _norm(name, T, H, x, residual=True):
    return {"name": name, "kind": "norm", "T": T, "H": H, "x": x, "residual": residual}


def _cache(kind, name, seqs, q_len, kv_len, **k):
    c = {"name": name, "kind": kind, "seqs": seqs, "q_len": q_len, "kv_len": kv_len, "ragged": False, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0, "fmt": "e4m3", "mix": 1}
    c.update(k)
    return c


def listed():
    return [
        # the norm ahead of the expert layer in a speculative verification step: 6 draft tokens of a small model
        _norm("norm_verify", 6, 2048, "bf16"),
        # the norm behind the expert layer (whose output is fp32) in a decode step of 32 sequences
        _norm("norm_decode", 32, 4096, "f32"),
        # the same in a prefill step of 8192 tokens
        _norm("norm_prefill", 8192, 4096, "bf16"),
        # each of 128 decoding sequences writes its one new token
        _cache("append", "append_decode", 128, 1, 700, ragged=True, page=16),
        # a prefill step writes 8192 tokens of three prompts of different lengths
        _cache("append", "append_prefill", 3, 4096, 4096, ragged=True),
        # a shared prefix is read back for a consumer of bf16 keys and values
        _cache("read", "read_prefix", 4, 8191, 8191, ragged=True, page=16),
        # a decode step: 32 sequences of up to 8k tokens, one new token each
        _cache("attend", "attend_decode", 32, 1, 8192, ragged=True, page=64),
        # a decode step at long context with a 4-bit cache and few sequences
        _cache("attend", "attend_decode_long", 3, 1, 65536, page=128, fmt="e2m1"),
        # verification of 6 draft tokens for one user: latency
        _cache("attend", "attend_verify", 1, 6, 2051, heads=16, kv_heads=2),
        # a step that mixes decoding sequences with chunks of prompts, with a sliding window and small heads
        _cache("attend", "attend_mixed", 24, 700, 5000, ragged=True, heads=40, kv_heads=8, dim=64, page=16, window=2048, mix=3),
        # chunked prefill: 2048 new tokens behind 14336 that are in the cache
        _cache("attend", "attend_chunk", 1, 2048, 16384),
        # a prompt of 8192 tokens in one step
        _cache("attend", "attend_prefill", 1, 8192, 8192),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# key/value heads and query heads for each of them
GROUPS = ((1, 8), (1, 13), (2, 8), (2, 16), (4, 5), (4, 8), (8, 2), (8, 5), (8, 8), (10, 1))
DEAREST = 8192 * 8192 * 32 * 128  # (query, key) pairs, padded to the longest sequence, times all heads' elements


def draw(rng):
    kind = rng.choice(["norm", "norm", "append", "read", "attend", "attend", "attend", "attend"])
    if kind == "norm":
        c = _norm("", _spread(rng, 1, 8192), BLOCK * rng.choice([_spread(rng, 32, 95), _spread(rng, 97, 128)]),
                  rng.choice(["bf16", "f32"]), rng.random() < 0.8)
        del c["name"]
        return c
    kv_heads, group = rng.choice(GROUPS)
    c = {"ragged": rng.random() < 0.7, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128]),
         "page": rng.choice([16, 32, 64, 128]), "mix": rng.randrange(1 << 20)}
    if kind == "append":
        q = _spread(rng, 1, 2048)
        c = _cache(kind, "", max(1, min(128, _spread(rng, 1, 8192) // q)), q, q + _spread(rng, 1, 2048), **c)
    elif kind == "read":
        q = _spread(rng, 64, 8192)
        c = _cache(kind, "", max(1, min(32, 24576 // q)), q, q, fmt=rng.choice(["e4m3", "e4m3", "e2m1"]), **c)
    elif rng.random() < 0.5:  # decoding or verifying
        q, kv = rng.choice([1, 1, 1, 2, 4, 6]), _spread(rng, 64, 32768)
        c = _cache(kind, "", max(1, min(64, _spread(rng, 1, 262144) // kv)), q, kv + q, fmt=rng.choice(["e4m3", "e4m3", "e2m1"]),
                   window=rng.choice([0, 0, 0, 1024]), **c)
    else:  # chunks of prompts
        q = _spread(rng, 16, 4096)
        c = _cache(kind, "", max(1, min(8, 4096 // q)), q, q + rng.choice([0, 1]) * _spread(rng, 16, 12288),
                   fmt=rng.choice(["e4m3", "e4m3", "e2m1"]), window=rng.choice([0, 0, 0, 1000]), **c)
        while c["seqs"] * c["q_len"] * c["kv_len"] * c["heads"] * c["dim"] > DEAREST or work(c)["flops"] > 2 * DEAREST:
            c["q_len"], c["kv_len"] = c["q_len"] * 3 // 4, c["kv_len"] * 3 // 4
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    n, q_max, kv_max = case["seqs"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return [q_max] * n, [kv_max] * n
    rng = random.Random(case["mix"])
    q, kv = [], []
    for b in range(n):
        if case["kind"] == "read":
            q.append(rng.randint(1, q_max))
            kv.append(q[-1])
            continue
        if q_max > 16 and n > 4:  # decoding sequences among the chunks, and one place of the batch that is empty
            t = 0 if b == n // 2 else 1 if rng.random() < 0.6 else rng.randint(2, q_max)
        else:
            t = rng.randint(max(1, q_max // 2), q_max)
        q.append(t)
        kv.append(t + rng.randint(0, kv_max - t))
    q[0], kv[0] = q_max, kv_max
    return q, kv


# ------------------------------------------------------------------ inputs
def _pow2(e):
    """2^e in fp32, exactly, for whole e in -127 .. 127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, fmt):
    """x [..., D] fp32 -> MX codes (one byte for each element, E2M1 not yet packed) and scale bytes."""
    emax, top = (8, 448.0) if fmt == "e4m3" else (2, 6.0)
    g = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = g.abs().amax(-1)
    s = (torch.frexp(amax).exponent - 1 - emax).clamp(-127, 127)
    s = torch.where(amax > 0, s, torch.full_like(s, -127))
    q = (g * _pow2(-s.unsqueeze(-1))).clamp(-top, top).reshape(x.shape)
    if fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = q.abs()
        mag = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
        codes = (mag + 8 * torch.signbit(q)).to(torch.uint8)
    return codes, (s + 127).to(torch.uint8)


def _stored(x, fmt):
    """x as it lies in a cache: codes (E2M1 packed in pairs, the even element in the low half) and scales."""
    codes, scales = _quantise(x, fmt)
    if fmt == "e2m1":
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes.contiguous(), scales.contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["kind"] == "norm":
        T, H = case["T"], case["H"]
        x = normal(T, H) * (normal(H) * 0.5).exp()
        st = {"case": case, "x": x.to(torch.bfloat16) if case["x"] == "bf16" else x, "eps": 1e-6,
              "residual": (normal(T, H) * 3).to(torch.bfloat16) if case["residual"] else None,
              "weight": (1 + 0.2 * normal(H)).to(torch.bfloat16),
              "residual_out": torch.empty(T, H, dtype=torch.bfloat16, device=dev) if case["residual"] else None,
              "y": torch.empty(T, H, dtype=torch.bfloat16, device=dev),
              "codes": torch.empty(T, H, dtype=torch.uint8, device=dev), "scales": torch.empty(T, H // BLOCK, dtype=torch.uint8, device=dev)}
        return st

    q_lens, kv_lens = _lengths(case)
    T, D, P, Hk, Hq = sum(q_lens), case["dim"], case["page"], case["kv_heads"], case["heads"]
    per_seq = max(1, -(-max(kv_lens) // P))
    pages = case["seqs"] * per_seq + 3
    order = torch.randperm(pages, generator=g, device=dev)
    st = {"case": case, "page": P, "T": T, "max_q": max(q_lens), "max_kv": max(kv_lens), "scale": D ** -0.5,
          "block_table": order[: case["seqs"] * per_seq].reshape(case["seqs"], per_seq).to(torch.int32).contiguous(),
          "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device=dev),
          "q_starts": torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32, device=dev)}
    # keys have channels of different sizes and values have tokens of different sizes, as in trained models
    wide = (normal(Hk, 1, D) * 0.5).exp()
    st["k_codes"], st["k_scales"] = _stored(normal(pages, Hk, P, D) * wide, case["fmt"])
    st["v_codes"], st["v_scales"] = _stored(normal(pages, Hk, P, D) * (normal(pages, Hk, P, 1) * 0.3).exp(), case["fmt"])
    # queries, keys and values are slices of one projection's output
    qkv = normal(T, (Hq + 2 * Hk) * D).to(torch.bfloat16)
    st["q"] = qkv[:, : Hq * D].view(T, Hq, D)
    st["k"] = qkv[:, Hq * D : (Hq + Hk) * D].view(T, Hk, D)
    st["v"] = qkv[:, (Hq + Hk) * D :].view(T, Hk, D)
    if case["kind"] == "attend":
        st["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    if case["kind"] == "read":
        st["k_out"] = torch.empty(T, Hk, D, dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.empty(T, Hk, D, dtype=torch.bfloat16, device=dev)
    if own:
        from block_scaled_mx_gb300 import mxmoe as mx

        st["cache"] = mx.KVCache.of(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], D, case["fmt"])
        size = mx.mx_paged_attention_workspace_size(T, case["seqs"], Hq, Hk, D, st["max_q"]) if case["kind"] == "attend" else 256
        st["ws"] = mx.alloc_workspace(size)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    kind = st["case"]["kind"]
    if own:
        from block_scaled_mx_gb300 import mxmoe as mx

        if kind == "norm":
            mx.mx_add_rmsnorm(st["x"], st["weight"], st["eps"], residual=st["residual"], residual_out=st["residual_out"],
                              y=st["y"], codes=st["codes"], scales=st["scales"])
        elif kind == "append":
            mx.mx_kv_append(st["cache"], st["k"], st["v"], st["block_table"], st["kv_lens"], st["q_starts"], st["ws"])
        elif kind == "read":
            mx.mx_kv_read(st["cache"], st["block_table"], st["kv_lens"], st["q_starts"], st["k_out"], st["v_out"], st["ws"])
        else:
            mx.mx_paged_attention(st["q"], st["cache"], st["block_table"], st["kv_lens"], st["q_starts"], st["out"], st["ws"],
                                  scale=st["scale"], window=st["case"]["window"], max_q_len=st["max_q"], lse=st["lse"])
    else:
        {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[kind](st)
    if kind == "norm":
        return [st["residual_out"], st["y"], *_values(st["codes"], st["scales"])]
    if kind == "append":
        return [*_values(st["k_codes"], st["k_scales"]), *_values(st["v_codes"], st["v_scales"])]
    if kind == "read":
        return [st["k_out"], st["v_out"]]
    return [st["out"], st["lse"]]


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _plain_norm(st):
    z = st["x"].float()
    if st["residual"] is not None:
        z = z + st["residual"].float()
        st["residual_out"].copy_(z)
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + st["eps"]) * st["weight"].float()
    st["y"].copy_(y)
    codes, scales = _quantise(y, "e4m3")
    st["codes"].copy_(codes)
    st["scales"].copy_(scales)


def _slots(st):
    """Page and place in it of each of the T tokens: the last ones of their sequences."""
    starts, t = st["q_starts"].long(), torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    at = st["kv_lens"].long()[b] - (starts[b + 1] - t)
    return st["block_table"].long()[b, at // st["page"]], at % st["page"]


def _plain_append(st):
    page, at = _slots(st)
    for x, codes, scales in ((st["k"], st["k_codes"], st["k_scales"]), (st["v"], st["v_codes"], st["v_scales"])):
        c, s = _stored(x.float(), st["case"]["fmt"])
        codes[page, :, at] = c
        scales[page, :, at] = s


def _decoded(codes, scales, fmt):
    """fp32 values of codes [..., D or D/2] with scales [..., D/32]."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=codes.device)
        both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        v = table[both.int()]
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(scales.int().unsqueeze(-1) - 127)).flatten(-2)


def _plain_read(st):
    page, at = _slots(st)
    fmt = st["case"]["fmt"]
    st["k_out"].copy_(_decoded(st["k_codes"][page, :, at], st["k_scales"][page, :, at], fmt))
    st["v_out"].copy_(_decoded(st["v_codes"][page, :, at], st["v_scales"][page, :, at], fmt))


def _plain_attend(st):
    case, T = st["case"], st["T"]
    B, Hq, Hk, D = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    G, mq, mk = Hq // Hk, st["max_q"], st["max_kv"]
    starts, kv = st["q_starts"].long(), st["kv_lens"].long()
    n = starts[1:] - starts[:-1]
    # the sequences side by side, padded to the longest
    j = torch.arange(mk, device="cuda")
    page = st["block_table"].long()[:, j // st["page"]]
    at = (j % st["page"]).expand(B, mk)
    here = (j < kv[:, None])[:, :, None, None]
    k = torch.where(here, _decoded(st["k_codes"][page, :, at], st["k_scales"][page, :, at], case["fmt"]), 0.0)
    v = torch.where(here, _decoded(st["v_codes"][page, :, at], st["v_scales"][page, :, at], case["fmt"]), 0.0)
    i = torch.arange(mq, device="cuda")
    row = (starts[:-1, None] + i).clamp(max=T - 1)
    q = st["q"][row].float().view(B, mq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * mq, D)
    s = (q @ k.permute(0, 2, 3, 1) * st["scale"]).view(B, Hk, G, mq, mk)
    last = (kv - n)[:, None] + i  # the last key that each query sees
    seen = (j <= last[:, :, None]) & (j < kv[:, None, None])
    if case["window"]:
        seen &= j > last[:, :, None] - case["window"]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = p.view(B, Hk, G * mq, mk) @ v.permute(0, 2, 1, 3)
    o = o.view(B, Hk, G, mq, D) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).squeeze(-1)
    real = i < n[:, None]
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[real].reshape(T, Hq, D))
    st["lse"].copy_(lse.permute(0, 3, 1, 2)[real].reshape(T, Hq))


# ------------------------------------------------------------------ what it costs, and what is exact
def work(case):
    if case["kind"] == "norm":
        n = case["T"] * case["H"]
        read = n * (2 if case["x"] == "bf16" else 4) + (2 * n if case["residual"] else 0) + 2 * case["H"]
        write = (2 * n if case["residual"] else 0) + 2 * n + n + n // BLOCK
        return {"bytes": read + write, "flops": 8 * n}
    q_lens, kv_lens = _lengths(case)
    D, Hk, Hq = case["dim"], case["kv_heads"], case["heads"]
    row = (D if case["fmt"] == "e4m3" else D // 2) + D // BLOCK  # bytes of one token's key or value of one head
    T = sum(q_lens)
    if case["kind"] in ("append", "read"):
        return {"bytes": 2 * T * Hk * (2 * D + row), "flops": 6 * T * Hk * D}
    pairs = keys = 0
    for n, kv in zip(q_lens, kv_lens):
        w = case["window"] or kv
        pairs += sum(min(w, kv - n + i + 1) for i in range(n))
        keys += min(kv, w + n - 1) if n else 0
    return {"bytes": 2 * keys * Hk * row + T * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    """The same from the definitions in 64 bits, one sequence and one head at a time."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    f64 = torch.float64
    if case["kind"] == "norm":
        z = st["x"].to(f64) + (0 if st["residual"] is None else st["residual"].to(f64))
        y = z / torch.sqrt((z ** 2).sum(1, keepdim=True) / case["H"] + st["eps"]) * st["weight"].to(f64)
        codes, scales = _exact_codes(y)
        return [z if st["residual"] is not None else None, y, codes, scales]
    fmt, P, D = case["fmt"], case["page"], case["dim"]
    starts, kv_lens, table = st["q_starts"].tolist(), st["kv_lens"].tolist(), st["block_table"].long()
    if case["kind"] == "append":
        k_codes, k_scales = (t.to(f64) for t in _values(st["k_codes"], st["k_scales"]))
        v_codes, v_scales = (t.to(f64) for t in _values(st["v_codes"], st["v_scales"]))
        for b, kv in enumerate(kv_lens):
            if starts[b] == starts[b + 1]:
                continue
            pos = torch.arange(kv - (starts[b + 1] - starts[b]), kv, device="cuda")
            page, at = table[b][pos // P], pos % P
            for x, c, s in ((st["k"], k_codes, k_scales), (st["v"], v_codes, v_scales)):
                c[page, :, at], s[page, :, at] = _exact_codes(x[starts[b] : starts[b + 1]].to(f64))
        return [k_codes, k_scales, v_codes, v_scales]

    def rows(codes, scales, b, pos):
        """[positions, heads, D] of a sequence."""
        page, at = table[b][pos // P], pos % P
        c, s = codes[page, :, at], scales[page, :, at]
        if fmt == "e4m3":
            sign, e, m = 1.0 - 2.0 * (c >> 7).to(f64), ((c >> 3) & 15).to(f64), (c & 7).to(f64)
            x = sign * torch.where(e > 0, (8 + m) * _exact_pow2(e - 10), m * 2.0 ** -9)
        else:
            x = torch.empty(*c.shape[:-1], D, dtype=f64, device=c.device)
            x[..., 0::2], x[..., 1::2] = c & 15, c >> 4
            e, m = (x % 8 // 2), x % 2
            x = torch.where(x >= 8, -1.0, 1.0) * torch.where(e > 0, (2 + m) * _exact_pow2(e - 2), m * 0.5)
        return x * _exact_pow2(s.to(f64) - 127).repeat_interleave(BLOCK, -1)

    if case["kind"] == "read":
        outs = []
        for codes, scales in ((st["k_codes"], st["k_scales"]), (st["v_codes"], st["v_scales"])):
            outs.append(torch.cat([rows(codes, scales, b, torch.arange(kv - (starts[b + 1] - starts[b]), kv, device="cuda")) for b, kv in enumerate(kv_lens)]))
        return outs
    G = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["T"], case["heads"], D, dtype=f64, device="cuda")
    lse = torch.full((st["T"], case["heads"]), -math.inf, dtype=f64, device="cuda")
    for b, kv in enumerate(kv_lens):
        n = starts[b + 1] - starts[b]
        if not n or not kv:
            continue
        pos = torch.arange(kv, device="cuda")
        K, V = rows(st["k_codes"], st["k_scales"], b, pos), rows(st["v_codes"], st["v_scales"], b, pos)
        last = torch.arange(kv - n, kv, device="cuda")[:, None]
        hidden = pos > last
        if case["window"]:
            hidden |= pos <= last - case["window"]
        for h in range(case["heads"]):
            q = st["q"][starts[b] : starts[b + 1], h].to(f64)
            s = (q @ K[:, h // G].T * st["scale"]).masked_fill_(hidden, -math.inf)
            lse[starts[b] : starts[b + 1], h] = torch.logsumexp(s, -1)
            out[starts[b] : starts[b + 1], h] = torch.softmax(s, -1) @ V[:, h // G]
    return [out, lse]


def _exact_codes(x):
    """E4M3 values and scales of x [..., D] in 64 bits: the nearest, an even code where two are as near."""
    g = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = g.abs().amax(-1, keepdim=True)
    s = torch.floor(torch.log2(top))
    s = torch.where(top > 0, s, -127.0)
    s = torch.where(_exact_pow2(s) > top, s - 1, s)
    s = torch.where(_exact_pow2(s + 1) <= top, s + 1, s) - 8
    s = torch.where(top > 0, s, -127.0).clamp(-127, 127)
    q = g / _exact_pow2(s)
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    e = torch.where(_exact_pow2(e + 1) <= q.abs(), e + 1, e).clamp(min=-6)
    step = _exact_pow2(e - 3)
    v = (torch.round(q / step) * step).clamp(-448, 448)
    return v.reshape(x.shape), _exact_pow2(s).squeeze(-1)


def _exact_pow2(e):
    """2^e in 64 bits for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
