"""Host-side argument checks of the operators that close a decoding step: every call
below is refused, or has nothing to do, before any device work (no GPU needed)."""
import ctypes
import decimal
import math

import pytest
import torch

import serve_reference as srv


@pytest.fixture(scope="module")
def L():
    from block_scaled_mx_gb300 import build as B
    from block_scaled_mx_gb300 import mxmoe as mx

    B.build()
    return mx.lib()


P = ctypes.c_void_p
fake = P(4096)   # never dereferenced
odd = P(4098)


# ------------------------------------------------------------------ projections
def test_linear_refusals(L):
    size = L.mx_linear_workspace_size(4, 100, 256, 0)
    assert size > 256 + 4 * 256 and L.mx_linear_workspace_size(0, 100, 256, 0) == 256

    def call(x=fake, c=None, sc=None, act=0, w=fake, wf=0, bias=None, T=4, N=100, K=256, out=fake, ot=0, ws=fake, wb=size):
        return L.mx_linear(x, c, sc, act, w, wf, bias, T, N, K, out, ot, ws, wb, None)

    assert call(T=0) == 0
    for bad in (dict(x=None), dict(c=fake, sc=fake), dict(x=None, c=fake), dict(x=None, sc=fake), dict(sc=fake), dict(w=None), dict(out=None), dict(ws=None),
                dict(T=-1), dict(N=0), dict(K=0), dict(act=2), dict(wf=-1), dict(ot=3)):
        assert call(**bad) == 1, bad
    for bad in (dict(K=48), dict(K=2 ** 20 + 32), dict(N=2 ** 22 + 1), dict(T=2 ** 22 + 1), dict(act=1, wf=0)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=P(4104)), dict(x=None, c=P(4104), sc=fake), dict(w=P(4112)), dict(bias=odd), dict(out=P(4104)), dict(ws=P(4112))):
        assert call(**bad) == 3, bad
    assert call(wb=size - 1) == 4
    need = L.mx_linear_prepared_bytes(100, 96, 1)
    assert need == 128 * 128 + 2 * 512 and L.mx_linear_prepared_bytes(100, 100, 1) == 0 and L.mx_linear_prepared_bytes(129, 160, 0) == 4 * (16384 + 512)

    def lay(c=fake, sc=fake, N=100, K=96, f=1, d=fake, db=need):
        return L.mx_linear_prepare(c, sc, N, K, f, d, db, None)

    for bad, want in ((dict(c=None), 1), (dict(sc=None), 1), (dict(d=None), 1), (dict(N=0), 1), (dict(f=2), 1), (dict(K=100), 2), (dict(c=P(4104)), 3),
                      (dict(d=P(4112)), 3), (dict(db=need - 1), 4)):
        assert lay(**bad) == want, bad


# ------------------------------------------------------------------ sandwich norm
def test_sandwich_refusals(L):
    def call(x=fake, xt=0, pw=fake, pt=0, gate=None, gt=0, kind=0, act=0, res=fake, rt=0, rs=1.0, bs=1.0, w=fake, wt=0, T=4, H=64,
             eps=1e-6, ro=fake, y=fake, fmt=0, codes=fake, scales=fake):
        return L.mx_sandwich_rmsnorm(x, xt, pw, pt, gate, gt, kind, act, res, rt, rs, bs, w, wt, T, H, eps, ro, y, fmt, codes, scales, None)

    assert call(T=0) == 0
    for bad in (dict(x=None), dict(res=None), dict(ro=None), dict(T=-1), dict(H=0), dict(xt=2), dict(rt=-1), dict(wt=5), dict(pt=3), dict(eps=0.0),
                dict(eps=math.nan), dict(rs=math.inf), dict(bs=math.nan), dict(fmt=2), dict(scales=None), dict(codes=None),
                dict(y=None, codes=None, scales=None), dict(w=None), dict(w=None, y=None), dict(kind=4, gate=fake), dict(kind=1), dict(gate=fake),
                dict(kind=-1), dict(act=2), dict(kind=3, gate=fake, gt=2)):
        assert call(**bad) == 1, bad
    for bad in (dict(H=48), dict(H=32800)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=odd), dict(res=odd), dict(w=odd), dict(pw=odd), dict(ro=odd), dict(y=odd), dict(codes=odd), dict(kind=1, gate=odd),
                dict(kind=3, gate=odd), dict(kind=2, gate=odd, gt=1), dict(kind=2, gate=P(4097))):
        assert call(**bad) == 3, bad


# ------------------------------------------------------------------ rotary positions
def _table(L, R=64, base=10000.0, scaling=0, factor=1.0, low=1.0, high=4.0, length=4096):
    out, amp = (ctypes.c_uint64 * max(R // 2, 1))(), ctypes.c_float()
    st = L.mx_rope_table(R, base, scaling, factor, low, high, length, ctypes.addressof(out), ctypes.addressof(amp))
    return st, list(out), amp.value


def test_rope_table_refusals(L):
    out = ctypes.addressof((ctypes.c_uint64 * 32)())
    assert L.mx_rope_table(64, 1e4, 0, 1.0, 1.0, 4.0, 0, None, out) == 1 and L.mx_rope_table(64, 1e4, 0, 1.0, 1.0, 4.0, 0, out, None) == 1
    for bad in (dict(R=0), dict(R=-2), dict(R=3), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=5), dict(scaling=-1),
                dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.nan), dict(scaling=2, R=2, factor=2.0), dict(scaling=3, length=0),
                dict(scaling=4, length=-1), dict(scaling=3, low=0.0), dict(scaling=3, low=4.0), dict(scaling=4, high=math.inf)):
        assert _table(L, **bad)[0] == 1, bad
    for fine in (dict(), dict(factor=math.nan, low=math.nan), dict(scaling=1, factor=1.0, length=0), dict(R=2)):
        assert _table(L, **fine)[0] == 0, fine


@pytest.mark.parametrize("scaling,name", list(enumerate(["none", "linear", "ntk", "yarn", "bands"])))
@pytest.mark.parametrize("R,base,factor,length,low,high", [(64, 10000.0, 8.0, 4096, 1.0, 32.0), (128, 500000.0, 16.0, 8192, 1.0, 4.0), (32, 10000.0, 1.0, 2048, 0.5, 2.0)])
def test_rope_table_values(L, scaling, name, R, base, factor, length, low, high):
    st, turns, amp = _table(L, R, base, scaling, factor, low, high, length)
    f, want_amp = srv.frequencies(R, base, name, factor, length, low, high)
    assert st == 0 and abs(amp - want_amp) <= 2.0 ** -24 * want_amp
    for got, x in zip(turns, f):
        x = x / (2 * math.pi)
        # a handful of roundings in 64 bits, each 2^-53; the exponent of a power by up to 14 of
        # them; the table holds whole multiples of 2^-64, rounded down
        assert abs(got / 2.0 ** 64 - x) <= 64 * 2.0 ** -53 * x + 2.0 ** -64


def _cache(**kw):
    from block_scaled_mx_gb300 import mxmoe as mx

    f = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, num_pages=8, page_size=16, n_kv_heads=2, head_dim=64, fmt=0)
    f.update(kw)
    return mx.KVCacheTables(*(f[n] for n, _ in mx.KVCacheTables._fields_))


def test_rope_append_refusals(L):
    def call(c=None, q=fake, qs=512, nq=8, qo=fake, os=512, k=fake, ks=512, v=fake, vs=512, pos=None, turns=fake, R=64, layout=0, amp=1.0, bt=fake,
             kv=fake, st=fake, n=2, mp=4, T=4, ws=fake, wb=256):
        c = _cache() if c is None else c
        return L.mx_rope_kv_append(ctypes.addressof(c), q, qs, nq, qo, os, k, ks, v, vs, pos, turns, R, layout, amp, bt, kv, st, n, mp, T, ws, wb, None)

    assert call(T=0) == 0 and call(n=0) == 0
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(turns=None), dict(bt=None), dict(kv=None), dict(st=None), dict(ws=None),
                dict(nq=-1), dict(nq=0), dict(qs=511), dict(os=100), dict(ks=127), dict(vs=1), dict(R=-16), dict(R=80), dict(layout=2),
                dict(amp=math.nan), dict(amp=math.inf), dict(T=-1), dict(n=-1), dict(mp=0), dict(c=_cache(fmt=2)), dict(c=_cache(num_pages=0))):
        assert call(**bad) == 1, bad
    for bad in (dict(R=24), dict(c=_cache(head_dim=288), qs=4096, os=4096, ks=4096, vs=4096), dict(c=_cache(head_dim=80), R=16, qs=4096, os=4096, ks=4096, vs=4096),
                dict(nq=20000, qs=2 ** 21, os=2 ** 21), dict(c=_cache(page_size=2 ** 30))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=odd), dict(qo=odd), dict(k=odd), dict(v=odd), dict(qs=516), dict(os=516), dict(ks=516), dict(vs=516), dict(pos=P(4097)),
                dict(turns=P(4100)), dict(ws=P(4112)), dict(bt=odd)):
        assert call(**bad) == 3, bad
    assert call(wb=255) == 4


# ------------------------------------------------------------------ sampling
def test_sample_refusals(L):
    def call(x=fake, type=0, stride=100, T=4, V=100, tau=None, k=None, p=None, m=None, u=fake, tok=fake, lp=None, ws=fake, wb=256):
        return L.mx_sample(x, type, stride, T, V, tau, k, p, m, u, tok, lp, ws, wb, None)

    assert call(T=0) == 0
    for bad in (dict(x=None), dict(u=None), dict(tok=None), dict(ws=None), dict(type=2), dict(stride=99), dict(T=-1), dict(V=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(V=800001, stride=10 ** 6), dict(V=400001, stride=10 ** 6, type=1), dict(T=2 ** 30)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=P(4097)), dict(x=odd, type=1), dict(tau=odd), dict(k=odd), dict(p=odd), dict(m=odd), dict(u=odd), dict(tok=odd), dict(lp=odd),
                dict(ws=P(4112))):
        assert call(**bad) == 3, bad
    assert call(wb=255) == 4
    assert L.mx_sample_workspace_size(-1, 5) == 0 and L.mx_sample_workspace_size(3, 0) == 0 and L.mx_sample_workspace_size(0, 5) == 256


# ------------------------------------------------------------------ the binding
def test_binding_checks_tensors(L):
    from block_scaled_mx_gb300 import mxmoe as mx

    meta = dict(device="meta")
    x, row = torch.empty(4, 64, **meta), torch.empty(64, **meta)
    with pytest.raises(ValueError, match="gate"):
        mx.mx_sandwich_rmsnorm(x, None, 1e-6, x, x, gate=torch.empty(4, **meta))
    with pytest.raises(ValueError, match="post_weight"):
        mx.mx_sandwich_rmsnorm(x, torch.empty(32, **meta), 1e-6, x, x)
    with pytest.raises(KeyError):
        mx.mx_sandwich_rmsnorm(x, None, 1e-6, x, x, gate_act="relu")
    with pytest.raises(KeyError):
        mx.Rope(64, layout="other", device="cpu")
    with pytest.raises(KeyError):
        mx.Rope(64, scaling="other", device="cpu")
    with pytest.raises(mx.MxError):
        mx.Rope(63, device="cpu")
    with pytest.raises(ValueError):
        mx.Rope(0, device="cpu")
    rope = mx.Rope(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    assert rope.turns.dtype == torch.int64 and rope.turns.shape == (32,) and abs(rope.amplitude - 1.138629436) < 1e-6
    logits = torch.empty(4, 50, **meta)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mx_sample(logits, row, row, row)
    with pytest.raises(ValueError, match="dense"):
        mx.mx_sample(logits.t(), row, row, row)


def test_binding_refuses_tensors_of_another_device(L, monkeypatch):
    """The stream is the current device's: a tensor that lies on another one is refused."""
    from block_scaled_mx_gb300 import mxmoe as mx

    class There:   # a tensor of cuda:1, of which a machine with one GPU has none
        is_cuda, device = True, "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        mx._here(There(), "x")
    monkeypatch.setattr(mx, "_current_device", lambda: 1)
    mx._here(There(), "x")


# ------------------------------------------------------------------ workspaces of captured graphs
def test_capture_refusals(L):
    from block_scaled_mx_gb300 import mxmoe as mx

    assert L.mx_capture_id(None, None) == 1
    assert L.mx_exchange_capture_mode(None) == 1
    for bad in (-1, 3):
        assert L.mx_exchange_capture_mode(ctypes.addressof(ctypes.c_int(bad))) == 1
    if not torch.cuda.is_available():
        assert mx.current_capture() == 0


class Gpu(torch.Tensor):
    """Host memory that says it lies on a GPU: for calls that are refused before they read it."""
    is_cuda = property(lambda t: True)

    def get_device(self):
        return self.gpu


def _gpu(shape, dtype=torch.float32, gpu=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Gpu)
    t.gpu = gpu
    return t


BF16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def _linear_call(mx, at):
    w = object.__new__(mx.LinearWeights)
    w.fmt, w.N, w.K, w.data = 0, 128, 256, at("w", (1024,), U8)
    return lambda: mx.mx_linear(w, at("out", (4, 128)), at("ws", (4096,), U8), codes=at("codes", (4, 256), U8), scales=at("scales", (4, 8), U8),
                                bias=at("bias", (128,)))


def _linear_x_call(mx, at):
    w = object.__new__(mx.LinearWeights)
    w.fmt, w.N, w.K, w.data = 0, 128, 256, at("w", (1024,), U8)
    return lambda: mx.mx_linear(w, at("out", (4, 128)), at("ws", (4096,), U8), x=at("x", (4, 256), BF16))


def _weights_call(mx, at):
    return lambda: mx.LinearWeights(at("codes", (128, 256), U8), at("scales", (128, 8), U8), "e4m3")


def _sandwich_call(mx, at):
    return lambda: mx.mx_sandwich_rmsnorm(at("x", (4, 64)), at("post_weight", (64,)), 1e-6, at("residual", (4, 64)), at("residual_out", (4, 64)),
                                          gate=at("gate", (64,)), weight=at("weight", (64,)), y=at("y", (4, 64), BF16), codes=at("codes", (4, 64), U8),
                                          scales=at("scales", (4, 2), U8))


def _rope_call(mx, at):
    cache = mx.KVCache.of(*(at("cache", (8, 2, 16, n), U8) for n in (64, 2, 64, 2)), 64)
    rope = mx.Rope(64, device="cpu")
    rope.turns = at("turns", (32,), torch.int64)
    return lambda: mx.mx_rope_kv_append(cache, rope, at("q", (4, 8, 64), BF16), at("k", (4, 2, 64), BF16), at("v", (4, 2, 64), BF16),
                                        at("block_table", (2, 4), I32), at("kv_lens", (2,), I32), at("q_starts", (3,), I32), at("ws", (256,), U8),
                                        q_out=at("q_out", (4, 8, 64), BF16), positions=at("positions", (4,), I32))


def _sample_call(mx, at):
    return lambda: mx.mx_sample(at("logits", (4, 50)), at("u", (4,)), at("tokens", (4,), I32), at("ws", (256,), U8), temperature=at("temperature", (4,)),
                                top_k=at("top_k", (4,), I32), top_p=at("top_p", (4,)), min_p=at("min_p", (4,)), logp=at("logp", (4,)))


@pytest.mark.parametrize("call", [_linear_call, _linear_x_call, _weights_call, _sandwich_call, _rope_call, _sample_call])
def test_binding_refuses_every_tensor_of_another_device(L, monkeypatch, call):
    from block_scaled_mx_gb300 import mxmoe as mx

    class NoLibrary:
        def __getattr__(self, name):
            def called(*a):
                raise AssertionError(f"{name} was called")

            return called

    def run(gpu_of):
        names = []
        with monkeypatch.context() as m:
            m.setattr(mx, "_current_device", lambda: 0)
            m.setattr(mx, "_current_raw_stream", lambda device: 0)
            make = call(mx, lambda name, *a: names.append(name) or _gpu(*a, gpu=gpu_of(name)))
            m.setattr(mx, "lib", NoLibrary)
            make()
        return names

    names = []
    with pytest.raises(AssertionError, match="was called"):     # all in place: on to the library
        run(lambda name: names.append(name) or 0)
    for other in sorted(set(names)):
        with pytest.raises(ValueError, match=f"^{other}: on .* but the current"):
            run(lambda name: int(name == other))


def _dec_turns(R, base, scaling, factor, low, high, length):
    """The table's formulas in 60 decimal digits: turns a position of each pair."""
    D = decimal.Decimal
    pi = D("3.14159265358979323846264338327950288419716939937510582097494")
    base, factor, low, high, length = D(base), D(factor), D(low), D(high), D(length)
    if scaling == "ntk":
        base *= factor ** (D(R) / (R - 2))
    out = []
    at = {t: R * (length / (2 * pi * t)).ln() / (2 * base.ln()) for t in (low, high)}
    first, last = max(math.floor(at[high]), 0), min(math.ceil(at[low]), R - 1)
    for i in range(R // 2):
        f, slow = base ** (D(-2 * i) / R), D(0)
        if scaling == "linear":
            slow = D(1)
        elif scaling == "yarn":
            slow = D(i - first) / max(D(last - first), D("0.001"))
        elif scaling == "bands":
            slow = 1 - (length * f / (2 * pi) - low) / (high - low)
        slow = min(max(slow, D(0)), D(1))
        out.append((f / factor * slow + f * (1 - slow)) / (2 * pi))
    return out


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("R,base,factor,length,low,high", [(16, 10000.0, 2.0, 4096, 1.0, 32.0), (64, 1e6, 3.0, 8192, 1.0, 4.0),
                                                           (128, 500000.0, 16.0, 32768, 0.5, 2.0), (256, 1.5, 1.0, 100, 1.0, 8.0), (256, 1e9, 7.0, 2048, 1.0, 32.0)])
def test_rope_table_is_near_enough_for_far_positions(L, scaling, R, base, factor, length, low, high):
    """What the header says of an angle: the table is at most 2^-52 turns a position off."""
    with decimal.localcontext() as c:
        c.prec = 60
        st, turns, _ = _table(L, R, base, ["none", "linear", "ntk", "yarn", "bands"].index(scaling), factor, low, high, length)
        want = _dec_turns(R, base, scaling, factor, low, high, length)
        assert st == 0
        # in units of 2^-53 of f_i <= 1: the power (2: an ulp), its exponent's rounding (x log(base)
        # base^-x <= 1 / e of one), its base's (ntk: 3), the mix (3, and 6 half f_i for a ramp with
        # high / (high - low) <= 4 / 3), 2 pi and the division by it (2): 10 at most in one scaling,
        # 10 / (2 pi) 2^-53 < 2^-52 turns, and what is cut off behind 2^-64
        assert max(abs(decimal.Decimal(t) / 2 ** 64 - w) for t, w in zip(turns, want)) <= decimal.Decimal(2) ** -52
