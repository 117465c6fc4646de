"""GPU parity of the sandwich norm (mx_sandwich_rmsnorm) and of rotary positions on the
way into the cache (mx_rope_kv_append) against plain fp64 references."""
import pytest
import torch

from block_scaled_mx_gb300 import mxmoe as mx

import block_reference as ref
import serve_reference as srv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------ sandwich norm
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ULP = 2.0 ** -24
# a sum of squares (each of H <= 32768 terms goes through at most 64 + 10 additions, the
# root halves it), mean, eps, root and two products
NORM_REL = 64 * ULP


def _gate(kind, T, H, g):
    shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(kind)
    return None if shape is None else 1 + torch.randn(*shape, generator=g)


def _sandwich(x, pw, eps, res, gate, act, bs, rs, w):
    """(z, its error bound, y, its error bound) in fp64."""
    n = x.double()
    rel = 4 * ULP
    if pw is not None:
        n = n / torch.sqrt((n * n).mean(1, keepdim=True) + eps) * pw.double()
        rel += NORM_REL
    if gate is not None:
        a = gate.double()
        if act == "sigmoid":
            a = torch.sigmoid(a)
            rel += 2.0 ** -20      # the fast exponential (2 ulp beside |g| 2^-24, |g| < 8) and division (2 ulp)
        n = n * a
    z = rs * res.double() + bs * n
    dz = rel * (bs * n).abs() + 2 * ULP * ((rs * res.double()).abs() + (bs * n).abs())
    if w is None:
        return z, dz, None, None
    inv = 1 / torch.sqrt((z * z).mean(1, keepdim=True) + eps)
    y = z * inv * w.double()
    moved = torch.sqrt((dz * dz).mean(1, keepdim=True)) * inv   # of the root, relative
    return z, dz, y, dz * inv * w.double().abs() + (NORM_REL + moved) * y.abs()


def _check(out, want, slack):
    step = torch.finfo(out.dtype).eps / 2
    assert torch.all((out.cpu().double() - want).abs() <= step * want.abs() + (1 + step) * slack)


@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (1, 2048), (7, 4096), (33, 4128), (2, 8192), (3, 8224), (2, 16416), (5, 32768)])
@pytest.mark.parametrize("xt,rt,wt,gate,act,post,fmt", [("bf16", "bf16", "bf16", None, "none", True, "e4m3"),
                                                        ("f32", "bf16", "f32", "full", "none", True, "e4m3"),
                                                        ("bf16", "f32", "bf16", "token", "sigmoid", False, "e2m1"),
                                                        ("f32", "f32", "bf16", "channel", "none", True, "e2m1"),
                                                        ("bf16", "bf16", "f32", "full", "sigmoid", True, "e2m1")])
def test_sandwich(T, H, xt, rt, wt, gate, act, post, fmt):
    g = torch.Generator().manual_seed(T * H)
    x = (torch.randn(T, H, generator=g) * 2).to(DT[xt])
    res = (torch.randn(T, H, generator=g) * 3).to(DT[rt])
    pw = (1 + 0.3 * torch.randn(H, generator=g)).to(DT[wt]) if post else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(DT[wt])
    gt = _gate(gate, T, H, g)
    gt = None if gt is None else gt.to(DT[xt])
    ro = torch.empty_like(res, device="cuda")
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(T, H // 2 if fmt == "e2m1" else H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    bs, rs, eps = 1.25, 0.8125, 1e-5      # the scales are exact in fp32
    mx.mx_sandwich_rmsnorm(x.cuda(), None if pw is None else pw.cuda(), eps, res.cuda(), ro, gate=None if gt is None else gt.cuda(),
                           gate_act=act, block_scale=bs, residual_scale=rs, weight=w.cuda(), y=y, codes=codes, scales=scales, fmt=fmt)
    z, dz, yd, dy = _sandwich(x, pw, eps, res, gt, act, bs, rs, w)
    _check(ro, z, dz)
    _check(y, yd, dy)
    assert srv.codes_hold(codes, scales, yd, dy, fmt) > 0.99


def test_sandwich_outputs_alone_and_in_place():
    T, H = 19, 1056
    g = torch.Generator().manual_seed(5)
    x, res = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w, gate = (torch.randn(H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    y, y2, ro, ro2 = (torch.empty_like(x) for _ in range(4))
    codes, codes2 = (torch.empty(T, H, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, scales2 = (torch.empty(T, H // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    kw = dict(gate=gate, block_scale=0.5)
    mx.mx_sandwich_rmsnorm(x, w, 1e-5, res, ro, weight=w, y=y, codes=codes, scales=scales, **kw)
    mx.mx_sandwich_rmsnorm(x, w, 1e-5, res, ro2, **kw)                 # no norm behind it
    assert torch.equal(ro2, ro)
    r2 = res.clone()
    mx.mx_sandwich_rmsnorm(x, w, 1e-5, r2, r2, weight=w, y=y2, **kw)
    assert torch.equal(r2, ro) and torch.equal(y2, y)
    x2 = x.clone()
    mx.mx_sandwich_rmsnorm(x2, w, 1e-5, res, x2, weight=w, codes=codes2, scales=scales2, **kw)
    assert torch.equal(x2, ro) and torch.equal(codes2, codes) and torch.equal(scales2, scales)


def test_sandwich_without_its_extras_is_the_residual_norm():
    T, H = 40, 2048
    g = torch.Generator().manual_seed(6)
    x, res = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.randn(H, generator=g).to(torch.bfloat16).cuda()
    outs = []
    for call in (lambda ro, **k: mx.mx_sandwich_rmsnorm(x, None, 1e-6, res, ro, weight=w, **k),
                 lambda ro, **k: mx.mx_add_rmsnorm(x, w, 1e-6, residual=res, residual_out=ro, **k)):
        for fmt in ("e4m3", "e2m1"):
            ro, y = torch.empty_like(x), torch.empty_like(x)
            codes = torch.empty(T, H // (1 if fmt == "e4m3" else 2), dtype=torch.uint8, device="cuda")
            scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
            call(ro, y=y, codes=codes, scales=scales, fmt=fmt)
            outs.append((ro, y, codes, scales))
    for a, b in zip(outs[:2], outs[2:]):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_sandwich_rows_of_zeros_and_gates_far_out():
    """A row of zeros stays zero, a sigmoid gate's ends are 0 and 1, a closed gate leaves the residual."""
    T, H = 4, 512
    x = torch.ones(T, H)
    x[0] = 0
    res = torch.full((T, H), 2.0)
    res[0] = 0
    gate = torch.zeros(T, 1)
    gate[1], gate[2], gate[3] = -200.0, 200.0, -87.5
    one = torch.ones(H, device="cuda")
    ro = torch.empty(T, H, device="cuda")
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    mx.mx_sandwich_rmsnorm(x.cuda(), one, 1e-6, res.cuda(), ro, gate=gate.cuda(), gate_act="sigmoid", weight=one, y=y, codes=codes, scales=scales)
    assert torch.all(ro[0] == 0) and torch.all(y[0] == 0) and torch.all(codes[0] == 0) and torch.all(scales[0] == 0)
    assert torch.all(ro[1] == 2) and torch.all(ro[3] == 2)
    assert torch.all((ro[2] - 3).abs() < 1e-5)


# ------------------------------------------------------------------ rotary positions
def _rope_inputs(T, hq, hk, D, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, (hq + 2 * hk) * D, generator=g) * 2).to(torch.bfloat16).cuda()   # slices of one projection
    return (qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D), qkv[:, (hq + hk) * D:].view(T, hk, D))


# the angle (2^-25 turns), sine and cosine (2 ulp each), amplitude, two products and a sum
ROPE_REL = 6.3 * 2.0 ** -25 + 5 * ULP


def _rope_check(q, k, v, q_out, cache, batch, pos, fmt, R, layout, f, amp):
    want, size = srv.rotate(q.cpu().double(), pos, f, amp, R, layout)
    _check(q_out, want, ROPE_REL * size)
    if layout == "half":
        assert torch.equal(q_out[..., R:], q[..., R:])
    tables = {n: getattr(cache, n).cpu() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    wk, sk = srv.rotate(k.cpu().double(), pos, f, amp, R, layout)
    for b, n in enumerate(batch.n):
        rows = slice(batch.starts[b], batch.starts[b] + n)
        page, at = batch.places(b, torch.arange(batch.kv[b] - n, batch.kv[b]))
        for x, size, c, s in ((wk, ROPE_REL * sk, "k_codes", "k_scales"), (v.cpu().double(), torch.zeros_like(sk), "v_codes", "v_scales")):
            assert srv.codes_hold(tables[c][page, :, at], tables[s][page, :, at], x[rows], size[rows], fmt) is not None, (b, c)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R,hq,hk,page,fmt", [(128, 128, 8, 2, 16, "e4m3"), (64, 64, 5, 1, 32, "e2m1"), (96, 48, 3, 3, 16, "e4m3"),
                                                (256, 64, 2, 2, 64, "e2m1"), (32, 16, 40, 10, 16, "e4m3"), (64, 32, 33, 11, 16, "e4m3"),
                                                (128, 112, 1, 1, 16, "e2m1"), (256, 256, 7, 1, 16, "e4m3")])
def test_rope(layout, D, R, hq, hk, page, fmt):
    batch = ref.make_batch([1, 5, 17, 2], [100, 5, 33, 4097], page, D + R)
    q, k, v = _rope_inputs(batch.T, hq, hk, D, R)
    cache = mx.KVCache(batch.pages, page, hk, D, fmt)
    rope = mx.Rope(R, layout=layout)
    q_out = torch.empty(batch.T, hq, D, dtype=torch.bfloat16, device="cuda")
    ws = mx.alloc_workspace(256)
    mx.mx_rope_kv_append(cache, rope, q, k, v, *batch.device(), ws, q_out=q_out)
    assert mx.moe_get_status(ws) == 0
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(batch.n, batch.kv)])
    f, amp = srv.frequencies(R)
    _rope_check(q, k, v, q_out, cache, batch, pos, fmt, R, layout, f, amp)
    # in place, and through many tokens at once: the same bits
    before = [getattr(cache, n).clone() for n in ("k_codes", "k_scales", "v_codes", "v_scales")]
    q2 = q.clone(memory_format=torch.contiguous_format)
    mx.mx_rope_kv_append(cache, rope, q2, k, v, *batch.device(), ws, q_out=q2)
    assert torch.equal(q2, q_out)
    assert all(torch.equal(a, getattr(cache, n)) for a, n in zip(before, ("k_codes", "k_scales", "v_codes", "v_scales")))


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
                                        ("yarn", dict(factor=16.0, original_length=4096)), ("bands", dict(factor=8.0, original_length=8192)),
                                        ("yarn", dict(factor=40.0, original_length=4096, low=2.0, high=20.0))])
def test_rope_scaled_and_far(scaling, kw):
    """Positions of up to 2^30, by `positions`: what is written stays where the lengths say."""
    R = D = 128
    batch = ref.make_batch([9], [9], 16, 3)
    q, k, v = _rope_inputs(9, 4, 2, D, 1)
    cache = mx.KVCache(batch.pages, 16, 2, D)
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 131071, 10 ** 7 + 3, 2 ** 30 - 1, -5, 77, 4096], dtype=torch.int32)
    rope = mx.Rope(R, base=500000.0, scaling=scaling, **kw)
    q_out = torch.empty(9, 4, D, dtype=torch.bfloat16, device="cuda")
    ws = mx.alloc_workspace(256)
    mx.mx_rope_kv_append(cache, rope, q, k, v, *batch.device(), ws, q_out=q_out, positions=pos.cuda())
    assert mx.moe_get_status(ws) == 0
    f, amp = srv.frequencies(R, 500000.0, scaling, kw["factor"], kw.get("original_length", 0), kw.get("low", 1.0),
                             kw.get("high", 32.0 if scaling == "yarn" else 4.0))
    assert abs(rope.amplitude - amp) <= 2.0 ** -23 * amp
    # p f in 64 bits is itself off by 2^-52 p f_i, at most 2^-22 at 2^30
    want, size = srv.rotate(q.cpu().double(), pos, f, amp, R, "half")
    _check(q_out, want, (ROPE_REL + 2.0 ** -21) * size)
    table = cache.k_codes.cpu()
    page, at = batch.places(0, torch.arange(9))
    wk, sk = srv.rotate(k.cpu().double(), pos, f, amp, R, "half")
    assert srv.codes_hold(table[page, :, at], cache.k_scales.cpu()[page, :, at], wk, (ROPE_REL + 2.0 ** -21) * sk, "e4m3") is not None


def test_rope_append_without_rotation_is_the_append():
    """At position 0 the angle is 0: codes are mx_kv_append's bit for bit, and q passes."""
    for fmt in ("e4m3", "e2m1"):
        batch = ref.make_batch([70, 1, 300], [70, 5, 310], 16, 8)
        q, k, v = _rope_inputs(batch.T, 4, 2, 64, 2)
        caches = [mx.KVCache(batch.pages, 16, 2, 64, fmt) for _ in range(3)]
        ws, q_out = mx.alloc_workspace(256), torch.empty(batch.T, 4, 64, dtype=torch.bfloat16, device="cuda")
        mx.mx_kv_append(caches[0], k, v, *batch.device(), ws)
        mx.mx_rope_kv_append(caches[1], mx.Rope(64), q, k, v, *batch.device(), ws, q_out=q_out,
                             positions=torch.zeros(batch.T, dtype=torch.int32, device="cuda"))
        mx.mx_rope_kv_append(caches[2], mx.Rope(32), None, k, v, *batch.device(), ws,
                             positions=torch.zeros(batch.T, dtype=torch.int32, device="cuda"))
        assert mx.moe_get_status(ws) == 0 and torch.equal(q_out, q)
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)) and torch.equal(getattr(caches[0], n), getattr(caches[2], n))


def test_rope_many_tokens_equal_few():
    """A large step splits its tokens over warps differently: the same bits as one token at a time."""
    batch = ref.make_batch([2500, 700], [2500, 900], 64, 4)
    q, k, v = _rope_inputs(batch.T, 8, 4, 128, 3)
    rope, ws = mx.Rope(128, layout="interleaved"), mx.alloc_workspace(256)
    one = mx.KVCache(batch.pages, 64, 4, 128)
    table, lens, starts = batch.device()
    q_out = torch.empty(batch.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    mx.mx_rope_kv_append(one, rope, q, k, v, table, lens, starts, ws, q_out=q_out)
    for t, b, pos in ((0, 0, 0), (1234, 0, 1234), (2499, 0, 2499), (2500, 1, 200), (3199, 1, 899)):
        other, o = mx.KVCache(batch.pages, 64, 4, 128), torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
        mx.mx_rope_kv_append(other, rope, q[t:t + 1], k[t:t + 1], v[t:t + 1], table[b:b + 1], torch.tensor([pos + 1], dtype=torch.int32, device="cuda"),
                             torch.tensor([0, 1], dtype=torch.int32, device="cuda"), ws, q_out=o)
        assert torch.equal(o[0], q_out[t])
        page, at = int(batch.table[b, pos // 64]), pos % 64
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(other, n)[page, :, at], getattr(one, n)[page, :, at])
    assert mx.moe_get_status(ws) == 0


def test_rope_leaves_padding_and_bad_metadata_alone():
    """Tokens past the last sequence, without a place or a page: nothing of theirs is written."""
    n, kv, page = [2, 3, 1], [2, 2, 40], 16       # the second has a token before its sequence
    batch = ref.make_batch(n, [2, 40, 40], page, 1)
    batch.table[2] = batch.pages + 5              # pages that do not exist
    T = batch.T + 4
    q, k, v = _rope_inputs(T, 2, 1, 64, 5)
    cache = mx.KVCache(batch.pages, page, 1, 64)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(cache, name).fill_(0x5A)
    q_out = torch.full((T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = mx.alloc_workspace(256)
    table, _, starts = batch.device()
    mx.mx_rope_kv_append(cache, mx.Rope(64), q, k, v, table, torch.tensor(kv, dtype=torch.int32, device="cuda"), starts, ws, q_out=q_out)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    written = [0, 1, 3, 4]
    for t in range(T):
        assert (not torch.all(q_out[t] == 7)) == (t in written), t
    places = {(int(batch.table[b, p // page]), p % page) for b, p in ((0, 0), (0, 1), (1, 0), (1, 1))}
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        t = getattr(cache, name).cpu()
        for pg in range(batch.pages):
            for at in range(page):
                if (pg, at) not in places:
                    assert torch.all(t[pg, :, at] == 0x5A)


def test_rope_in_a_graph_on_another_stream():
    batch = ref.make_batch([1] * 5, [30, 1, 17, 64, 2], 16, 6)
    q, k, v = _rope_inputs(5, 4, 2, 64, 9)
    rope, ws = mx.Rope(64), mx.alloc_workspace(256)
    want, got = (mx.KVCache(batch.pages, 16, 2, 64) for _ in range(2))
    dev = batch.device()
    o, p = torch.empty(5, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    mx.mx_rope_kv_append(want, rope, q, k, v, *dev, ws, q_out=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_rope_kv_append(got, rope, q, k, v, *dev, ws, q_out=p)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, p) and torch.equal(want.k_codes, got.k_codes) and torch.equal(want.v_codes, got.v_codes)


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
@pytest.mark.parametrize("gt", ["bf16", "f32"])
def test_sigmoid_of_far_gates_in_fp32(kind, gt):
    """A residual of zeros in fp32 leaves act(gate) x alone: the sigmoid has to be as good as
    fp32 wherever its gate lies."""
    T, H = 401, 128
    x = torch.ones(T, H) * 0.75
    far = torch.linspace(-86.0, 20.0, T)   # the result is a normal number for all of them
    gate = {"channel": torch.linspace(-86.0, 20.0, H), "token": far[:, None], "full": far[:, None] + torch.linspace(-1, 1, H)}[kind].to(DT[gt])
    res, ro = torch.zeros(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    mx.mx_sandwich_rmsnorm(x.cuda(), None, 1e-6, res, ro, gate=gate.cuda(), gate_act="sigmoid")
    want = torch.sigmoid(gate.double()) * x.double()
    # the exponential (a power of two, 2 ulp: 2^-22, and its correction, 2^-24), a sum (2^-24), a
    # division (2 ulp: 2^-22), two products (2^-24 each)
    assert torch.all((ro.cpu().double() - want).abs() <= (2 * 2.0 ** -22 + 4 * 2.0 ** -24) * want)
