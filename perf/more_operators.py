"""The rest of a decoding step, from hidden states to tokens, as cases that can be timed and compared.

Four operators, which a decoder model calls one after the other:

  linear   a dense projection with MX weights: the activations are quantised, then multiplied (``mx_linear``)
  rope     rotary positions for new queries and keys, keys and values quantised into a paged MX cache (``mx_rope_kv_append``)
  norm     norm behind a block, its gate and scale, the residual, the norm ahead of the next block (``mx_sandwich_rmsnorm``)
  sample   a token from logits, by temperature, top-k, top-p and min-p from a given random number (``mx_sample``)

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
def _linear(name, T, K, N, w, act="e4m3", out="bf16", bias=False):
    return {"name": name, "kind": "linear", "T": T, "K": K, "N": N, "w": w, "act": act, "out": out, "bias": bias}


def _rope(name, seqs, q_len, past, **k):
    c = {"name": name, "kind": "rope", "seqs": seqs, "q_len": q_len, "past": past, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "page": 64, "mix": 1}
    c.update(k)
    return c


def _norm(name, T, H, x="bf16", gate="none", post=True, y=True):
    return {"name": name, "kind": "norm", "T": T, "H": H, "x": x, "gate": gate, "post": post, "y": y}


def _sample(name, T, V, logits, rules, spread):
    return {"name": name, "kind": "sample", "T": T, "V": V, "logits": logits, "rules": rules, "spread": spread}


def listed():
    return [
        # the query, key and value projection of a few decoding sequences, 4-bit weights: latency and weight streaming
        _linear("linear_decode", 4, 4096, 6144, "e2m1"),
        # the output projection for the draft tokens of some sequences, 8-bit weights
        _linear("linear_verify", 96, 4096, 4096, "e4m3"),
        # logits of a decode step of 32 sequences over a vocabulary of an odd size
        _linear("linear_head", 32, 4096, 100003, "e2m1", out="f32"),
        # a projection of a prefill step of 8192 tokens, 4 bits on both sides
        _linear("linear_prefill", 8192, 4096, 6144, "e2m1", act="e2m1", bias=True),
        # 128 decoding sequences, one new token each
        _rope("rope_decode", 128, 1, 700, page=16),
        # a prefill step of 8192 tokens of three prompts, neighbouring elements paired, half of the head rotated
        _rope("rope_prefill", 3, 4096, 0, layout="interleaved", rot=64),
        # a chunk of 2048 tokens far into a long context whose frequencies are scaled
        _rope("rope_long", 1, 2048, 500000, scaling="yarn", page=128),
        # behind the attention in a decode step of 32 sequences
        _norm("norm_decode", 32, 4096),
        # behind the experts (whose output is fp32) in a prefill step of 8192 tokens, a gate for each element
        _norm("norm_prefill", 8192, 4096, x="f32", gate="full"),
        # one sequence's next token: latency
        _sample("sample_one", 1, 100003, "f32", "all", 2.5),
        # a batch whose requests all have rules of their own
        _sample("sample_batch", 64, 100003, "f32", "mixed", 2.5),
        # a large batch of a large vocabulary, logits in 16 bits
        _sample("sample_large", 256, 131072, "bf16", "mixed", 2.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# key/value heads and query heads for each of them
GROUPS = ((1, 8), (1, 13), (2, 8), (4, 5), (4, 8), (8, 4), (8, 5), (10, 1))
DEAREST = 8192 * 4096 * 6144


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear", "rope", "rope", "norm", "sample", "sample"])
    if kind == "linear":
        w = rng.choice(["e4m3", "e2m1"])
        act = rng.choice(["e4m3", "e4m3", "e2m1"]) if w == "e2m1" else "e4m3"
        K = BLOCK * _spread(rng, 8, 256)
        if rng.random() < 0.25:  # a vocabulary
            T, N = _spread(rng, 1, 64), _spread(rng, 16384, 131072)
        else:
            T, N = _spread(rng, 1, 8192), _spread(rng, 128, 16384)
        while T * K * N > DEAREST:
            T = T * 3 // 4
        c = _linear("", max(T, 1), K, N, w, act, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3)
    elif kind == "rope":
        kv_heads, group = rng.choice(GROUPS)
        q, dim = _spread(rng, 1, 4096), rng.choice([64, 96, 128, 128, 256])
        c = _rope("", max(1, min(128, _spread(rng, 1, 8192) // q)), q, rng.choice([0, _spread(rng, 16, 100000)]), heads=kv_heads * group,
                  kv_heads=kv_heads, dim=dim, rot=rng.choice([32, dim // 2, dim, dim]), layout=rng.choice(["half", "interleaved"]),
                  scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 20))
    elif kind == "norm":
        c = _norm("", _spread(rng, 1, 8192), BLOCK * _spread(rng, 16, 128), rng.choice(["bf16", "f32"]),
                  rng.choice(["none", "channel", "token", "full", "sigmoid"]), rng.random() < 0.8, rng.random() < 0.8)
    else:
        V = _spread(rng, 2000, 200000)
        c = _sample("", max(1, min(_spread(rng, 1, 512), 256 * 131072 // V)), V, rng.choice(["f32", "bf16"]),
                    rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]), rng.uniform(1.0, 4.0))
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    rng, q, kv = random.Random(case["mix"]), [], []
    for b in range(case["seqs"]):
        q.append(case["q_len"] if b == 0 else rng.randint(max(1, case["q_len"] // 4), case["q_len"]))
        kv.append(q[-1] + (case["past"] if b == 0 else rng.randint(case["past"] // 2, case["past"])))
    return q, kv


def _frequencies(case):
    """Turns of the angle for one position, of each pair, and the rotation's amplitude."""
    R, base, factor, length = case["rot"], 10000.0, 16.0, 32768
    kind, amp = case["scaling"], 1.0
    if kind == "ntk":
        base *= factor ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "yarn":  # slow pairs are slowed down, fast ones stay, a ramp over the pairs between
        at = [R * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(R // 2)]
        f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
        amp = 0.1 * math.log(factor) + 1.0
    elif kind == "bands":  # the same by wavelengths, the ramp over the turns in the original length
        out = []
        for x in f:
            turns = length * x / (2 * math.pi)
            smooth = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append((1 - smooth) * x / factor + smooth * x)
        f = out
    return f, amp


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
        mag = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
        codes = mag + 8 * torch.signbit(q).to(torch.uint8)
    return codes, (s + 127).to(torch.uint8)


def _decoded(codes, scales, fmt):
    """fp32 values of codes [..., D], one byte each, with scales [..., D/32]."""
    v = codes.view(torch.float8_e4m3fn).float() if fmt == "e4m3" else torch.tensor(E2M1 + tuple(-m for m in E2M1), device=codes.device)[codes.int()]
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(scales.int().unsqueeze(-1) - 127)).flatten(-2)


def prepare(case, seed):
    dev, kind = "cuda", case["kind"]
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    bf16 = torch.bfloat16
    if kind == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        # activations with channels of different sizes, as behind a norm
        st = {"case": case, "x": (normal(T, K) * (normal(K) * 0.5).exp()).to(bf16),
              "out": torch.empty(T, N, dtype=bf16 if case["out"] == "bf16" else torch.float32, device=dev),
              "bias": normal(N) if case["bias"] else None}
        codes, st["w_scales"] = _quantise(normal(N, K) * K ** -0.5 * (normal(N, 1) * 0.3).exp(), case["w"])
        st["w_codes"] = codes if case["w"] == "e4m3" else codes[:, 0::2] | (codes[:, 1::2] << 4)
        if own:  # weights are laid out once, and the workspace is kept
            from block_scaled_mx_gb300 import mxmoe as mx

            st["w"] = mx.LinearWeights(st["w_codes"], st["w_scales"], case["w"])
            st["ws"] = mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, K, case["act"]))
        return st
    if kind == "rope":
        q_lens, kv_lens = _lengths(case)
        T, D, P, Hk, Hq = sum(q_lens), case["dim"], case["page"], case["kv_heads"], case["heads"]
        # pages are held for the new tokens alone: what lies before them is other sequences' business
        per_seq = max(-(-n // P) for n in kv_lens)
        kept = [(kv - 1) // P - (kv - q) // P + 1 for q, kv in zip(q_lens, kv_lens)]
        order = torch.randperm(sum(kept) + 3, generator=g, device=dev).to(torch.int32)
        table, at = torch.zeros(case["seqs"], per_seq, dtype=torch.int32, device=dev), 0
        for b, n in enumerate(kept):
            first = (kv_lens[b] - q_lens[b]) // P
            table[b, first : first + n] = order[at : at + n]
            at += n
        f, amp = _frequencies(case)
        # queries, keys and values are slices of one projection's output
        qkv = normal(T, (Hq + 2 * Hk) * D).to(bf16)
        st = {"case": case, "page": P, "T": T, "block_table": table, "amp": amp, "f": torch.tensor(f, dtype=torch.float64, device=dev),
              "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device=dev),
              "q_starts": torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32, device=dev),
              "q": qkv[:, : Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D : (Hq + Hk) * D].view(T, Hk, D), "v": qkv[:, (Hq + Hk) * D :].view(T, Hk, D),
              "q_out": torch.empty(T, Hq, D, dtype=bf16, device=dev)}
        shape = (sum(kept) + 3, Hk, P)
        for x in "kv":
            st[x + "_codes"] = torch.randint(0, 120, (*shape, D), generator=g, device=dev, dtype=torch.uint8)
            st[x + "_scales"] = torch.randint(110, 130, (*shape, D // BLOCK), generator=g, device=dev, dtype=torch.uint8)
        if own:
            from block_scaled_mx_gb300 import mxmoe as mx

            st["cache"] = mx.KVCache.of(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], D, "e4m3")
            st["rope"] = mx.Rope(case["rot"], layout=case["layout"], scaling=case["scaling"], factor=16.0, original_length=32768)
            st["ws"] = mx.alloc_workspace(256)
        return st
    if kind == "norm":
        T, H = case["T"], case["H"]
        x = normal(T, H) * (normal(H) * 0.5).exp()
        shape = {"channel": (H,), "token": (T, 1), "full": (T, H), "sigmoid": (T, H)}.get(case["gate"])
        return {"case": case, "x": x.to(bf16) if case["x"] == "bf16" else x, "eps": 1e-6, "residual_scale": 0.9, "block_scale": 1.3,
                "residual": (normal(T, H) * 3).to(bf16), "gate": None if shape is None else (1 + 0.5 * normal(*shape)).to(bf16),
                "post_weight": (1 + 0.2 * normal(H)).to(bf16) if case["post"] else None, "weight": (1 + 0.2 * normal(H)).to(bf16),
                "residual_out": torch.empty(T, H, dtype=bf16, device=dev), "y": torch.empty(T, H, dtype=bf16, device=dev) if case["y"] else None,
                "codes": torch.empty(T, H, dtype=torch.uint8, device=dev), "scales": torch.empty(T, H // BLOCK, dtype=torch.uint8, device=dev)}
    T, V, rules = case["T"], case["V"], case["rules"]
    logits = normal(T, V) * case["spread"]
    # some tokens are banned
    logits[torch.rand(T, V, generator=g, device=dev) < 0.01] = -math.inf

    def some(values, off, name):
        """One value a row, or the one that switches the rule off where a row does without it; None where none has it."""
        if rules not in (name, "all", "mixed"):
            return None
        return torch.where(torch.rand(T, generator=g, device=dev) < (0.7 if rules == "mixed" else 1.1), values, torch.full_like(values, off))

    def uniform():
        return torch.rand(T, generator=g, device=dev)

    st = {"case": case, "logits": logits.to(bf16) if case["logits"] == "bf16" else logits, "u": uniform(), "temperature": 0.5 + uniform(),
          "top_k": some(torch.randint(20, 1000, (T,), generator=g, device=dev, dtype=torch.int32), 0, "top_k"),
          "top_p": some(0.5 + 0.49 * uniform(), 1.0, "top_p"), "min_p": some(0.001 + 0.1 * uniform(), 0.0, "min_p"),
          "tokens": torch.empty(T, dtype=torch.int32, device=dev), "logp": torch.empty(T, dtype=torch.float32, device=dev)}
    if rules == "mixed":  # a few requests are greedy
        st["temperature"] = torch.where(uniform() < 0.1, 0.0, st["temperature"])
    if own:
        from block_scaled_mx_gb300 import mxmoe as mx

        st["ws"] = mx.alloc_workspace(mx.mx_sample_workspace_size(T, V))
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        from block_scaled_mx_gb300 import mxmoe as mx

        if kind == "linear":
            mx.mx_linear(st["w"], st["out"], st["ws"], x=st["x"], act_fmt=case["act"], bias=st["bias"])
        elif kind == "rope":
            mx.mx_rope_kv_append(st["cache"], st["rope"], st["q"], st["k"], st["v"], st["block_table"], st["kv_lens"], st["q_starts"], st["ws"],
                                 q_out=st["q_out"])
        elif kind == "norm":
            mx.mx_sandwich_rmsnorm(st["x"], st["post_weight"], st["eps"], st["residual"], st["residual_out"], gate=st["gate"],
                                   gate_act="sigmoid" if case["gate"] == "sigmoid" else "none", block_scale=st["block_scale"],
                                   residual_scale=st["residual_scale"], weight=st["weight"], y=st["y"], codes=st["codes"], scales=st["scales"])
        else:
            mx.mx_sample(st["logits"], st["u"], st["tokens"], st["ws"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                         min_p=st["min_p"], logp=st["logp"])
    else:
        {"linear": _plain_linear, "rope": _plain_rope, "norm": _plain_norm, "sample": _plain_sample}[kind](st)
    if kind == "linear":
        return st["out"]
    if kind == "rope":
        return [st["q_out"], *_values(st["k_codes"], st["k_scales"]), *_values(st["v_codes"], st["v_scales"])]
    if kind == "norm":
        return [st["residual_out"], *([st["y"]] if case["y"] else []), *_values(st["codes"], st["scales"])]
    return [st["tokens"], st["logp"]]


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _plain_linear(st):
    case = st["case"]
    a = _decoded(*_quantise(st["x"].float(), case["act"]), case["act"])
    codes = st["w_codes"]
    if case["w"] == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    out = a @ _decoded(codes, st["w_scales"], case["w"]).t()
    if st["bias"] is not None:
        out = out + st["bias"]
    st["out"].copy_(out)


def _places(st):
    """Position, page and place in it of each of the T tokens: the last ones of their sequences."""
    starts, t = st["q_starts"].long(), torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = st["kv_lens"].long()[b] - (starts[b + 1] - t)
    return pos, st["block_table"].long()[b, pos // st["page"]], pos % st["page"]


def _plain_rope(st):
    case = st["case"]
    R, half = case["rot"], case["layout"] == "half"
    pos, page, at = _places(st)
    angle = pos.double()[:, None] * st["f"]
    cos, sin = (torch.cos(angle) * st["amp"]).float()[:, None], (torch.sin(angle) * st["amp"]).float()[:, None]

    def rotated(x):
        x = x.float()
        a, b = (x[..., : R // 2], x[..., R // 2 : R]) if half else (x[..., 0:R:2], x[..., 1:R:2])
        a, b = a * cos - b * sin, a * sin + b * cos
        return torch.cat((torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2), x[..., R:]), -1)

    st["q_out"].copy_(rotated(st["q"]))
    for x, codes, scales in ((rotated(st["k"]), st["k_codes"], st["k_scales"]), (st["v"].float(), st["v_codes"], st["v_scales"])):
        codes[page, :, at], scales[page, :, at] = _quantise(x, "e4m3")


def _plain_norm(st):
    x = st["x"].float()
    if st["post_weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * st["post_weight"].float()
    if st["gate"] is not None:
        gate = st["gate"].float()
        x = x * (torch.sigmoid(gate) if st["case"]["gate"] == "sigmoid" else gate)
    z = st["residual"].float() * st["residual_scale"] + x * st["block_scale"]
    st["residual_out"].copy_(z)
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + st["eps"]) * st["weight"].float()
    if st["y"] is not None:
        st["y"].copy_(y)
    codes, scales = _quantise(y, "e4m3")
    st["codes"].copy_(codes)
    st["scales"].copy_(scales)


def _plain_sample(st):
    x = st["logits"].float()
    T, V = x.shape
    greedy = st["temperature"] == 0
    # in 64 bits: a weight's rounding moves the borders that the random number falls between
    z = (x.double() - x.amax(-1, keepdim=True).double()) / torch.where(greedy, 1.0, st["temperature"]).double()[:, None]
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = torch.exp(z)
    rank = torch.arange(V, device="cuda")
    keep = (rank < 1) | ~greedy[:, None]
    if st["top_k"] is not None:
        keep &= (rank < st["top_k"][:, None]) | (st["top_k"] <= 0)[:, None]
    if st["top_p"] is not None:
        mass = torch.cumsum(torch.where(keep, w, 0.0), -1)
        keep &= (mass - w < mass[:, -1:] * st["top_p"].double()[:, None]) | (st["top_p"] >= 1)[:, None]
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None]
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    mass = torch.cumsum(w, -1)
    token = (mass <= mass[:, -1:] * st["u"].double()[:, None]).sum(-1)
    st["tokens"].copy_(token)
    st["logp"].copy_(torch.log(w.gather(1, token[:, None])[:, 0] / mass[:, -1]))


# ------------------------------------------------------------------ what it costs, and what is exact
def work(case):
    kind = case["kind"]
    if kind == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        weights = N * K // (1 if case["w"] == "e4m3" else 2) + N * K // BLOCK
        return {"bytes": 2 * T * K + weights + T * N * (2 if case["out"] == "bf16" else 4) + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    if kind == "rope":
        T, D, Hk, Hq = sum(_lengths(case)[0]), case["dim"], case["kv_heads"], case["heads"]
        return {"bytes": T * (4 * Hq * D + 2 * Hk * (2 * D + D + D // BLOCK)), "flops": T * (3 * (Hq + Hk) * case["rot"] + 6 * Hk * D)}
    if kind == "norm":
        n, T, H = case["T"] * case["H"], case["T"], case["H"]
        gate = {"channel": H, "token": T, "full": n, "sigmoid": n}.get(case["gate"], 0)
        return {"bytes": n * (2 if case["x"] == "bf16" else 4) + 4 * n + 2 * gate + (2 * n if case["y"] else 0) + n + n // BLOCK + 4 * H, "flops": 14 * n}
    n = case["T"] * case["V"]
    return {"bytes": n * (4 if case["logits"] == "f32" else 2) + 24 * case["T"], "flops": 4 * n}


def exact(case, seed):
    """The same from the definitions in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    f64, kind = torch.float64, case["kind"]
    if kind == "linear":
        x = _exact_quantised(st["x"].to(f64), case["act"])
        out = torch.empty(case["T"], case["N"], dtype=f64, device="cuda")
        for n in range(0, case["N"], 8192):  # the weights of 8192 columns at a time
            out[:, n : n + 8192] = x @ _exact_values(st["w_codes"][n : n + 8192], st["w_scales"][n : n + 8192], case["w"]).T
        return out if st["bias"] is None else out + st["bias"].to(f64)
    if kind == "rope":
        pos, page, at = _places(st)
        f, amp = _frequencies(case)
        R, turn = case["rot"], pos.to(f64)[:, None] * torch.tensor(f, dtype=f64, device="cuda")
        turn = torch.polar(torch.full_like(turn, amp), turn)[:, None, :]

        def turned(x):
            x = x.to(f64).clone()
            if case["layout"] == "half":
                z = torch.complex(x[..., : R // 2], x[..., R // 2 : R]) * turn
                x[..., : R // 2], x[..., R // 2 : R] = z.real, z.imag
            else:
                z = torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous()) * turn
                x[..., :R] = torch.view_as_real(z).flatten(-2)
            return x

        outs = [turned(st["q"])]
        for x, codes, scales in ((turned(st["k"]), st["k_codes"], st["k_scales"]), (st["v"].to(f64), st["v_codes"], st["v_scales"])):
            c, s = (t.to(f64) for t in _values(codes, scales))
            c[page, :, at], s[page, :, at] = _exact_codes(x, "e4m3")
            outs += [c, s]
        return outs
    if kind == "norm":
        n = st["x"].to(f64)
        if case["post"]:
            n = n / torch.sqrt((n ** 2).sum(1, keepdim=True) / case["H"] + st["eps"]) * st["post_weight"].to(f64)
        if st["gate"] is not None:
            n = n * (1 / (1 + torch.exp(-st["gate"].to(f64))) if case["gate"] == "sigmoid" else st["gate"].to(f64))
        z = st["residual_scale"] * st["residual"].to(f64) + st["block_scale"] * n
        y = z / torch.sqrt((z ** 2).sum(1, keepdim=True) / case["H"] + st["eps"]) * st["weight"].to(f64)
        return [z, *([y] if case["y"] else []), *_exact_codes(y, "e4m3")]
    tokens, logp = [], []
    for t in range(case["T"]):  # one request at a time, over its candidates alone
        x = st["logits"][t].to(f64)
        tau = st["temperature"][t].item()
        best = torch.argsort(x, descending=True, stable=True)
        if tau == 0:
            best = best[:1]
        if st["top_k"] is not None and st["top_k"][t] > 0:
            best = best[: int(st["top_k"][t])]
        p = torch.softmax(x[best] / (tau or 1.0), 0)
        if st["top_p"] is not None and st["top_p"][t] < 1:
            before = torch.cumsum(p, 0) - p
            best = best[: int((before < st["top_p"][t].to(f64)).sum())]
        p = p[: len(best)]
        if st["min_p"] is not None:
            best = best[p >= st["min_p"][t].to(f64) * p[0]]
        best = torch.sort(best).values
        p = torch.softmax(x[best] / (tau or 1.0), 0)
        at = torch.searchsorted(torch.cumsum(p, 0), st["u"][t].to(f64), right=True).clamp(max=len(best) - 1)
        tokens.append(best[at])
        logp.append(torch.log(p[at]))
    return [torch.stack(tokens).to(torch.int32), torch.stack(logp)]


def _exact_pow2(e):
    """2^e in 64 bits for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(x, fmt):
    """Element values and scales of x [..., D] in 64 bits: the nearest, an even code where two are as near."""
    emax, low, bits, most = (8, -6, 3, 448.0) if fmt == "e4m3" else (2, 0, 1, 6.0)
    g = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = g.abs().amax(-1, keepdim=True)
    s = torch.frexp(top).exponent.to(torch.float64) - 1 - emax
    s = torch.where(top > 0, s, -127.0).clamp(-127, 127)
    q = g / _exact_pow2(s)
    e = (torch.frexp(q).exponent.to(torch.float64) - 1).clamp(min=low)
    step = _exact_pow2(e - bits)
    v = (torch.round(q / step) * step).clamp(-most, most)
    return v.reshape(x.shape), _exact_pow2(s).squeeze(-1)


def _exact_quantised(x, fmt):
    v, s = _exact_codes(x, fmt)
    return v * s.repeat_interleave(BLOCK, -1)


def _exact_values(c, s, fmt):
    """Values of codes as they are stored (E2M1 packed in pairs) with their scales, from the formats' bits."""
    if fmt == "e4m3":
        sign, e, m = 1.0 - 2.0 * (c >> 7).double(), ((c >> 3) & 15).double(), (c & 7).double()
        x = sign * torch.where(e > 0, (8 + m) * _exact_pow2(e - 10), m * 2.0 ** -9)
    else:
        x = torch.stack((c & 15, c >> 4), -1).flatten(-2).double()
        e, m = torch.floor(x % 8 / 2), x % 2
        x = torch.where(x >= 8, -1.0, 1.0) * torch.where(e > 0, (2 + m) * _exact_pow2(e - 2), m * 0.5)
    return x * _exact_pow2(s.double() - 127).repeat_interleave(BLOCK, -1)
