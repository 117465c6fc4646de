"""Plain fp64 references of the operators that close a decoding step, on the CPU,
written from the definitions in include/mxmoe.h, and the checks their tests share."""
import math

import torch

import block_reference as ref


def codes_hold(codes, scales, want, slack, fmt):
    """Whether MX codes are those of some value within `slack` of `want` (fp64 [..., D]):
    each scale that of a block maximum in that range, each element between the roundings
    of the range's ends (in blocks whose scale the range leaves no choice of).  Returns
    the share of such blocks, or None."""
    codes, scales = codes.cpu(), scales.cpu()
    lo, hi = (want.abs() - slack).clamp(min=0), want.abs() + slack
    s_lo, q_lo = ref.quantise(lo, fmt)
    s_hi, q_hi = ref.quantise(hi, fmt)
    if not torch.all((scales == s_lo) | (scales == s_hi)):
        return None
    sure = s_lo == s_hi
    v = ref.decode(codes, torch.full_like(scales, 127), fmt)
    ok = (v.abs() >= q_lo) & (v.abs() <= q_hi) & ((v == 0) | (torch.signbit(v) == torch.signbit(want)) | (want.abs() <= slack))
    return float(sure.double().mean()) if torch.all(ok.unflatten(-1, (-1, 32)) | ~sure.unsqueeze(-1)) else None


def frequencies(R, base=10000.0, scaling="none", factor=1.0, length=0, low=1.0, high=4.0):
    """(radians a position of each pair, amplitude)."""
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        d = [R * math.log(length / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low)]
        a, b = max(math.floor(d[0]), 0), min(math.ceil(d[1]), R - 1)
        share = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(R // 2)]
        return [x / factor * s + x * (1 - s) for x, s in zip(f, share)], 0.1 * math.log(factor) + 1
    if scaling == "bands":
        out = []
        for x in f:
            t = length * x / (2 * math.pi)
            s = 1.0 if t >= high else 0.0 if t <= low else (t - low) / (high - low)
            out.append(s * x + (1 - s) * x / factor)
        return out, 1.0
    return f, 1.0


def rotate(x, pos, f, amp, R, layout):
    """x [T, heads, D] fp64 at positions pos [T] -> rotated, and the sizes |a| + |b| that
    its error scales with."""
    out, size = x.clone(), x.abs()
    for i in range(R // 2):
        m, n = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c = torch.tensor([math.cos(p * f[i]) for p in pos.tolist()], dtype=torch.float64)[:, None]
        s = torch.tensor([math.sin(p * f[i]) for p in pos.tolist()], dtype=torch.float64)[:, None]
        out[..., m] = amp * (x[..., m] * c - x[..., n] * s)
        out[..., n] = amp * (x[..., m] * s + x[..., n] * c)
        size[..., m] = size[..., n] = amp * (x[..., m].abs() + x[..., n].abs())
    return out, size


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of its probability) of one row, by a sort in 64 bits; the last value
    is how near the draw came to another token: the distance of u to the token's border,
    in units of the whole mass."""
    x = [float(v) for v in logits]
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    order = [i for i in order if x[i] > -math.inf]
    if temperature == 0:
        return order[0], 0.0, 1.0
    top = x[order[0]]
    w = {i: 1.0 if x[i] == top else math.exp((x[i] - top) / temperature) for i in order}
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        total, before, kept = math.fsum(w[i] for i in order), 0.0, []
        for i in order:
            if before >= top_p * total and kept:
                break
            kept.append(i)
            before += w[i]
        order = kept
    order = sorted(i for i in order if w[i] >= min_p)
    total, run = math.fsum(w[i] for i in order), 0.0
    for i in order:
        if run + w[i] > u * total or i == order[-1]:
            return i, math.log(w[i] / total) if w[i] > 0 else -math.inf, min(abs(run - u * total), abs(run + w[i] - u * total)) / total
        run += w[i]
