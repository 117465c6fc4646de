"""Plain fp64 references of the operators around the expert layer, on the CPU,
and the error bounds their tests use.  Everything is written from the
definitions in include/mxmoe.h; sizes are small, so loops are fine."""
import math
from dataclasses import dataclass

import torch

BLOCK = 32
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _e4m3_table():
    v = []
    for c in range(128):
        e, m = c >> 3, c & 7
        v.append((8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9)
    v[127] = math.nan
    return torch.tensor(v + [-x for x in v], dtype=torch.float64)


E4M3 = _e4m3_table()


def decode(codes, scales, fmt):
    """fp64 values of code rows [..., D or D/2] with scale rows [..., D/32]."""
    if fmt == "e4m3":
        v = E4M3[codes.long()]
    else:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        v = E2M1[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127)
    return (v.unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def quantise(x, fmt):
    """Scale bytes and the nearest grid values (ties to the even code) of fp64 rows x [..., D]."""
    top = 448.0 if fmt == "e4m3" else 6.0
    emax = 8 if fmt == "e4m3" else 2
    grid = E4M3[:127] if fmt == "e4m3" else E2M1
    g = x.unflatten(-1, (-1, BLOCK))
    amax = g.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    s = torch.where(amax > 0, (e - emax).clamp(-127, 127), -127)
    q = (g * torch.pow(torch.tensor(2.0, dtype=torch.float64), -s.double()).unsqueeze(-1)).clamp(-top, top)
    a = q.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (s + 127).to(torch.uint8), (grid[pick] * torch.where(torch.signbit(q), -1.0, 1.0)).flatten(-2)


@dataclass
class Batch:
    """A paged batch on the CPU: n new and kv cached tokens of each sequence."""
    n: list
    kv: list
    page: int
    pages: int
    table: torch.Tensor

    @property
    def T(self):
        return sum(self.n)

    @property
    def starts(self):
        return [sum(self.n[:b]) for b in range(len(self.n) + 1)]

    def device(self):
        return (self.table.cuda(), torch.tensor(self.kv, dtype=torch.int32).cuda(),
                torch.tensor(self.starts, dtype=torch.int32).cuda())

    def places(self, b, pos):
        """(pages, offsets) of positions of sequence b."""
        return self.table[b].long()[pos // self.page], pos % self.page


def make_batch(n, kv, page, seed, spare=2):
    g = torch.Generator().manual_seed(seed)
    per = max(1, max(-(-k // page) for k in kv)) + 1
    pages = len(n) * per + spare
    table = torch.randperm(pages, generator=g)[: len(n) * per].reshape(len(n), per).to(torch.int32)
    return Batch(list(n), list(kv), page, pages, table)


def attention(q, k_codes, k_scales, v_codes, v_scales, fmt, batch, scale, causal, window):
    """(out, lse, bound of |out| errors, bound of lse errors), fp64.

    Bounds: out is rounded to bf16 (2^-8 relative); a softmax weight is rounded to
    f16 or bf16 for the second product (at most 2^-8, applied to sum p |v|);
    a score sums D exact products in fp32 (D * 2^-24 of sum |q k|), which moves
    every weight by that much and the sum by as much again; weights below
    2^-24 of the largest may be lost (2^-24 * max |v| a key)."""
    T, Hq, D = q.shape
    Hk = k_codes.shape[1]
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double()
    for b, (n, kv) in enumerate(zip(batch.n, batch.kv)):
        if n == 0 or kv == 0:
            continue
        page, at = batch.places(b, torch.arange(kv))
        K, V = decode(k_codes[page, :, at], k_scales[page, :, at], fmt), decode(v_codes[page, :, at], v_scales[page, :, at], fmt)
        for i in range(n):
            pos = kv - n + i
            hi = min(kv, pos + 1) if causal else kv
            lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                continue
            t = batch.starts[b] + i
            for h in range(Hq):
                k, v = K[lo:hi, h * Hk // Hq], V[lo:hi, h * Hk // Hq]
                s = k @ qd[t, h] * scale
                ds = float((k.abs() @ qd[t, h].abs()).max()) * scale * D * 2.0 ** -24 + 2.0 ** -20
                p = torch.softmax(s, 0)
                out[t, h] = p @ v
                lse[t, h] = torch.logsumexp(s, 0)
                spread = p @ v.abs()
                tol[t, h] = 2.0 ** -8 * out[t, h].abs() + (2.0 ** -8 + 3 * ds) * spread + 2.0 ** -24 * len(s) * v.abs().max()
                tol_lse[t, h] = 2 * ds + 2.0 ** -20 * (1 + abs(float(lse[t, h])))
    return out, lse, tol, tol_lse
