"""GPU parity of the residual norm with MX output (mx_add_rmsnorm) and of the
paged MX cache's writes and reads (mx_kv_append, mx_kv_read) against plain fp64
references."""
import pytest
import torch

from block_scaled_mx_gb300 import mxmoe as mx

import block_reference as ref

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


# ------------------------------------------------------------------ residual norm
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# fp32: z (2^-24), the sum of squares (each of H <= 32768 terms goes through at
# most 32 + 10 additions, and the root halves it), mean, eps, root and two products
NORM_REL = 64 * 2.0 ** -24


def _norm_check(x, res, w, eps, got_res, y, codes, scales, fmt):
    z = x.float() + (res.float() if res is not None else 0)
    if res is not None:
        assert torch.equal(got_res.cpu(), z.to(res.dtype))   # one fp32 addition, one rounding
    zd = x.double() + (res.double() if res is not None else 0)
    yd = zd / torch.sqrt((zd * zd).mean(1, keepdim=True) + eps) * w.double()
    # z itself is a rounded sum: relative to the operands where they cancel
    slack = NORM_REL * yd.abs()
    if res is not None:
        inv = 1 / torch.sqrt((zd * zd).mean(1, keepdim=True) + eps)
        slack = slack + 2.0 ** -24 * (x.double().abs() + res.double().abs()) * inv * w.double().abs()
    if y is not None:
        got = y.cpu().double()
        assert torch.all((got - yd).abs() <= 2.0 ** -8 * yd.abs() + 2 * slack)
    if codes is not None:
        lo, hi = yd.abs() - slack, yd.abs() + slack
        s_lo, q_lo = ref.quantise(lo.clamp(min=0), fmt)
        s_hi, q_hi = ref.quantise(hi, fmt)
        got_s = scales.cpu()
        assert torch.all((got_s == s_lo) | (got_s == s_hi))
        sure = s_lo == s_hi   # a block whose largest value lies on a power of two may take either scale
        v = ref.decode(codes.cpu(), torch.full_like(got_s, 127), fmt)
        ok = (v.abs() >= q_lo) & (v.abs() <= q_hi) & ((v == 0) | (torch.signbit(v) == torch.signbit(yd)) | (yd.abs() <= slack))
        assert torch.all(ok.unflatten(-1, (-1, 32)) | ~sure.unsqueeze(-1))
        return float(sure.double().mean())
    return 1.0


@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (1, 2048), (7, 4096), (33, 4128), (2, 8192), (3, 8224), (5, 32768)])
@pytest.mark.parametrize("xt,rt,wt,fmt", [("bf16", "bf16", "bf16", "e4m3"), ("f32", "bf16", "f32", "e4m3"),
                                          ("bf16", None, "bf16", "e2m1"), ("f32", "f32", "bf16", "e2m1")])
def test_add_rmsnorm(T, H, xt, rt, wt, fmt):
    g = torch.Generator().manual_seed(T * H)
    x = (torch.randn(T, H, generator=g) * 2).to(DT[xt])
    res = (torch.randn(T, H, generator=g) * 3).to(DT[rt]) if rt else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(DT[wt])
    eps = 1e-6
    ro = torch.empty_like(res, device="cuda") if rt else None
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(T, H // 2 if fmt == "e2m1" else H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    mx.mx_add_rmsnorm(x.cuda(), w.cuda(), eps, residual=None if res is None else res.cuda(), residual_out=ro, y=y,
                      codes=codes, scales=scales, fmt=fmt)
    assert _norm_check(x, res, w, eps, ro, y, codes, scales, fmt) > 0.99


def test_add_rmsnorm_outputs_alone_and_in_place():
    """y alone and codes alone equal the joint call's; residual_out may be the
    residual or x itself."""
    T, H = 19, 1056
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    res = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(H, generator=g).to(torch.bfloat16).cuda()
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    ro = torch.empty_like(x)
    codes, codes2 = (torch.empty(T, H, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, scales2 = (torch.empty(T, H // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    mx.mx_add_rmsnorm(x, w, 1e-5, residual=res, residual_out=ro, y=y, codes=codes, scales=scales)
    r2 = res.clone()
    mx.mx_add_rmsnorm(x, w, 1e-5, residual=r2, residual_out=r2, y=y2)
    assert torch.equal(r2, ro) and torch.equal(y2, y)
    x2 = x.clone()
    mx.mx_add_rmsnorm(x2, w, 1e-5, residual=res, residual_out=x2, codes=codes2, scales=scales2)
    assert torch.equal(x2, ro) and torch.equal(codes2, codes) and torch.equal(scales2, scales)


def test_add_rmsnorm_rows_of_zeros_and_of_one_spike():
    T, H = 4, 512
    x = torch.zeros(T, H)
    x[1, 77] = 1e4
    x[2] = 1e-30
    x[3] = 1e15
    w = torch.ones(H)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    mx.mx_add_rmsnorm(x.cuda(), w.cuda(), 1e-6, y=y, codes=codes, scales=scales)
    assert torch.all(y[0] == 0) and torch.all(codes[0] == 0) and torch.all(scales[0] == 0)
    _norm_check(x, None, w, 1e-6, None, y, codes, scales, "e4m3")


def test_add_rmsnorm_codes_feed_the_grouped_gemm():
    """The codes drive moe_grouped_gemm_swiglu as mx_quantize_act's would: with a
    unit weight and x already normalised they are its codes but for rows' rounding."""
    T, H = 8, 256
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    codes, c2 = (torch.empty(T, H, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, s2 = (torch.empty(T, H // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    mx.mx_add_rmsnorm(x, w, 1e-6, y=y, codes=codes, scales=scales)
    mx.mx_quantize_act(y, c2, s2)
    a, b = ref.decode(codes.cpu(), scales.cpu(), "e4m3"), ref.decode(c2.cpu(), s2.cpu(), "e4m3")
    # y's bf16 rounding moves a value by 2^-8, the two quantisations by a step of 2^-3 at most
    assert torch.all((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9 * torch.pow(2.0, s2.cpu().double() - 127).repeat_interleave(32, 1))
    assert float((a != b).double().mean()) < 0.1


# ------------------------------------------------------------------ the cache
def _kv_inputs(T, heads, dim, seed, fused):
    g = torch.Generator().manual_seed(seed)
    if fused:   # slices of one projection: the token stride is not the row
        qkv = (torch.randn(T, 3 * heads * dim, generator=g) * 2).to(torch.bfloat16).cuda()
        return qkv[:, heads * dim:2 * heads * dim].view(T, heads, dim), qkv[:, 2 * heads * dim:].view(T, heads, dim)
    k = (torch.randn(T, heads, dim, generator=g) * 2).to(torch.bfloat16)
    v = torch.randn(T, heads, dim, generator=g) * torch.exp(2 * torch.randn(T, heads, 1, generator=g))
    return k.cuda(), v.to(torch.bfloat16).cuda()


CACHE_CASES = [([1], [1], 16, 1, 64), ([3, 0, 5, 1], [3, 0, 40, 17], 16, 2, 128), ([50, 1, 33], [50, 100, 129], 48, 3, 64),
               ([130], [300], 64, 8, 128), ([7, 9], [7, 100], 5, 2, 96), ([1] * 70, list(range(1, 71)), 32, 1, 32)]


@pytest.mark.parametrize("n,kv,page,heads,dim", CACHE_CASES)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("fused", [False, True])
def test_kv_append_and_read(n, kv, page, heads, dim, fmt, fused):
    """Codes and scales are the quantiser's bit for bit at the tokens' places and
    every other place keeps what it held; reading gives the stored values."""
    batch = ref.make_batch(n, kv, page, 3)
    k, v = _kv_inputs(batch.T, heads, dim, 7, fused)
    cache = mx.KVCache(batch.pages, page, heads, dim, fmt)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xA5)
    ws = mx.alloc_workspace(256)
    dev = batch.device()
    mx.mx_kv_append(cache, k, v, *dev, ws)
    assert mx.moe_get_status(ws) == 0
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        row = dim // 2 if fmt == "e2m1" else dim
        want_c = torch.full((batch.pages, heads, page, row), 0xA5, dtype=torch.uint8)
        want_s = torch.full((batch.pages, heads, page, dim // 32), 0xA5, dtype=torch.uint8)
        flat = x.reshape(batch.T * heads, dim).contiguous()
        c = torch.empty(batch.T * heads, row, dtype=torch.uint8, device="cuda")
        s = torch.empty(batch.T * heads, dim // 32, dtype=torch.uint8, device="cuda")
        mx.mx_quantize_act(flat, c, s, fmt=fmt)
        rs, rq = ref.quantise(flat.cpu().double(), fmt)
        assert torch.equal(s.cpu(), rs)
        assert torch.equal(ref.decode(c.cpu(), torch.full_like(rs, 127), fmt), rq)
        for b in range(len(n)):
            if n[b] == 0:
                continue
            at, off = batch.places(b, torch.arange(kv[b] - n[b], kv[b]))
            sl = slice(batch.starts[b], batch.starts[b + 1])
            want_c[at, :, off] = c.cpu().view(batch.T, heads, row)[sl]
            want_s[at, :, off] = s.cpu().view(batch.T, heads, dim // 32)[sl]
        assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    ko, vo = (torch.empty(batch.T, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mx.mx_kv_read(cache, *dev, ko, vo, ws)
    assert mx.moe_get_status(ws) == 0
    for x, o in ((k, ko), (v, vo)):
        s, q = ref.quantise(x.reshape(-1, dim).cpu().double(), fmt)
        want = (q.unflatten(-1, (-1, 32)) * torch.pow(2.0, s.double() - 127).unsqueeze(-1)).flatten(-2)
        assert torch.equal(o.cpu().double().reshape(-1, dim), want)   # four significant bits at most: exact in bf16


def test_kv_read_whole_sequences():
    """With q_starts counting kv_lens the whole context comes back."""
    batch = ref.make_batch([9, 30], [9, 30], 16, 1)
    k, v = _kv_inputs(batch.T, 2, 64, 3, False)
    cache = mx.KVCache(batch.pages, 16, 2, 64)
    ws = mx.alloc_workspace(256)
    mx.mx_kv_append(cache, k, v, *batch.device(), ws)
    table, kv, _ = batch.device()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    mx.mx_kv_read(cache, table, kv, torch.tensor([0, 9, 39], dtype=torch.int32, device="cuda"), ko, vo, ws)
    _, q = ref.quantise(k.reshape(-1, 64).cpu().double(), "e4m3")
    assert float((ko.cpu().double().reshape(-1, 64) - k.cpu().double().reshape(-1, 64)).abs().max()) > 0
    assert torch.all((ko - k).abs() <= 2.0 ** -4 * k.abs() + 2.0 ** -3 * k.abs().amax(-1, keepdim=True))


def test_kv_extreme_scales():
    """Blocks of zeros, of bf16's subnormals and of its largest values."""
    x = torch.zeros(4, 1, 64)
    x[1, 0, :32] = 2.0 ** -130
    x[2, 0, 32:] = 3.0e38
    x[3, 0, 5] = -2.0 ** -133
    x = x.to(torch.bfloat16)
    batch = ref.make_batch([4], [4], 16, 1)
    for fmt in ("e4m3", "e2m1"):
        cache = mx.KVCache(batch.pages, 16, 1, 64, fmt)
        ws = mx.alloc_workspace(256)
        mx.mx_kv_append(cache, x.cuda(), x.cuda(), *batch.device(), ws)
        ko, vo = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
        mx.mx_kv_read(cache, *batch.device(), ko, vo, ws)
        s, q = ref.quantise(x.reshape(-1, 64).double(), fmt)
        want = (q.unflatten(-1, (-1, 32)) * torch.pow(torch.tensor(2.0, dtype=torch.float64), s.double() - 127).unsqueeze(-1)).flatten(-2)
        assert torch.equal(ko.cpu().reshape(-1, 64).double(), want.to(torch.bfloat16).double())


def test_kv_bad_metadata_is_reported_and_skipped():
    """A page id out of range, a length shorter than the new tokens and one past
    the table: reported, skipped, the other sequences written; padding rows are
    ignored by append and zero from read."""
    batch = ref.make_batch([2, 3, 2, 2], [20, 2, 2, 2], 16, 1)
    T = batch.T + 3   # padding rows
    k, v = _kv_inputs(T, 2, 64, 9, False)
    table, kv, starts = batch.device()
    table = table.clone()
    kv = kv.clone()
    table[0, 1] = batch.pages          # tokens 18, 19 of sequence 0 (position 18 is in page 1)
    kv[2] = 100000                     # past the table
    cache = mx.KVCache(batch.pages, 16, 2, 64)
    ws = mx.alloc_workspace(256)
    mx.mx_kv_append(cache, k, v, table, kv, starts, ws)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    mx.mx_kv_read(cache, table, kv, starts, ko, vo, ws)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    assert mx.moe_get_status(ws) == 0
    good = list(range(3, 5)) + [7, 8]  # two of sequence 1's three tokens have places, sequence 3's both
    for t in range(T):
        if t in good:
            assert torch.all((ko[t] - k[t]).abs() <= 2.0 ** -4 * k[t].abs() + 2.0 ** -3 * k[t].abs().amax())
            assert float(ko[t].abs().sum()) > 0
        else:
            assert float(ko[t].abs().sum()) == 0 and float(vo[t].abs().sum()) == 0


@pytest.mark.parametrize("starts,kv,good", [
    ([0, 2, 50], [20, 48], [0, 1]),        # the second sequence's end lies past the tokens
    ([-3, 2, 5], [20, 30], [2, 3, 4]),     # the first one's start is negative
    ([0, 2, 5], [33, 30], [2, 3, 4]),      # a length past the table, by one token
    ([0, 2, 5], [20, -1], [0, 1])])
def test_kv_starts_and_lengths_out_of_range(starts, kv, good):
    """A sequence whose start, end or length is out of range is left out as a whole,
    as the attention leaves it out: nothing of it is written, read or kept."""
    T, page = 5, 16
    k, v = _kv_inputs(T, 2, 64, 11, False)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    batch = (table, torch.tensor(kv, dtype=torch.int32, device="cuda"), torch.tensor(starts, dtype=torch.int32, device="cuda"))
    cache = mx.KVCache(4, page, 2, 64)
    ws = mx.alloc_workspace(256)
    mx.mx_kv_append(cache, k, v, *batch, ws)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    mx.mx_kv_read(cache, *batch, ko, vo, ws)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    written = cache.k_scales.amax(dim=(1, 3)) > 0
    assert int(written.sum()) == len(good)
    for t in range(T):
        for x, o in ((k, ko), (v, vo)):
            if t in good:
                # half a step of e4m3 (2^-4), or of the smallest of the block
                assert torch.all((o[t] - x[t]).abs().float() <= 2.0 ** -4 * x[t].abs().float() + 2.0 ** -3 * x[t].abs().amax().float())
                assert float(o[t].abs().sum()) > 0
            else:
                assert float(o[t].abs().sum()) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_kv_read_of_a_scale_that_is_nan(fmt):
    """A scale byte of 255 reads as NaN whatever the codes, zero among them."""
    batch = ref.make_batch([3], [3], 16, 1)
    k, v = _kv_inputs(3, 1, 64, 3, False)
    k[1, 0, 40] = 0.0
    cache = mx.KVCache(batch.pages, 16, 1, 64, fmt)
    ws = mx.alloc_workspace(256)
    mx.mx_kv_append(cache, k, v, *batch.device(), ws)
    ko, vo, ko2, vo2 = (torch.empty_like(k) for _ in range(4))
    mx.mx_kv_read(cache, *batch.device(), ko, vo, ws)
    page, at = batch.places(0, torch.tensor([1]))
    cache.k_scales[page[0], 0, at[0], 1] = 255
    mx.mx_kv_read(cache, *batch.device(), ko2, vo2, ws)
    hit = torch.zeros(3, 1, 64, dtype=torch.bool, device="cuda")
    hit[1, 0, 32:] = True
    assert torch.all(torch.isnan(ko2[hit])) and torch.equal(ko2[~hit], ko[~hit]) and torch.equal(vo2, vo)


def test_add_rmsnorm_e2m1_codes_feed_the_grouped_gemms():
    """MXFP4 codes of the norm through both grouped GEMMs, against the layer in one call
    on the values that the codes stand for, which it quantises to the same codes."""
    from block_scaled_mx_gb300 import block as B

    T, H, I, E, k = 37, 256, 128, 8, 2
    layer = B.random_block(H, I, E, k, 4, 2, 64, fmt="e2m1", seed=5).experts
    opts = mx.layer_opts(act_fmt="e2m1")
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    codes = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    mx.mx_add_rmsnorm(x, w, 1e-6, codes=codes, scales=scales, fmt="e2m1")
    values = ref.decode(codes.cpu(), scales.cpu(), "e2m1").to(torch.bfloat16).cuda()
    again, again_s = torch.empty_like(codes), torch.empty_like(scales)
    mx.mx_quantize_act(values, again, again_s, fmt="e2m1")
    assert torch.equal(again, codes) and torch.equal(again_s, scales)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, weights = torch.empty(T, k, **i32), torch.empty(T, k, dtype=torch.float32, device="cuda")
    mx.moe_route_topk(logits, k, ids, weights)
    counts, offsets, order = torch.empty(E + 1, **i32), torch.empty(E + 2, **i32), torch.empty(T * (k + 1), **i32)
    mx.moe_permute(ids, E, counts, offsets, order, mx.alloc_workspace(mx.moe_permute_workspace_size(T, E, k)))
    h = torch.empty(T * (k + 1), I // 2, dtype=torch.uint8, device="cuda")
    hs = torch.empty(T * (k + 1), I // 32, dtype=torch.uint8, device="cuda")
    ws = mx.alloc_workspace(mx.moe_gemm_workspace_size(T, H, I, E, k))
    sizes = (layer.fmt, T, H, I, E, k)
    mx.moe_grouped_gemm_swiglu_ex(codes, scales, offsets, order, layer.w1, *sizes, h, hs, ws, opts)
    out = torch.zeros(T, H, dtype=torch.float32, device="cuda")
    mx.moe_grouped_gemm_down_combine(h, hs, offsets, order, weights, layer.w2, *sizes, out, ws, opts=opts)
    assert mx.moe_get_status(ws) == 0
    one = layer.forward(values, logits, opts=opts)
    # an h next to a border may take either code, a step of at most 2^-1: one in 1000 of
    # them moves the output by 2^-1 / 1000^0.5 = 0.016 (relative, L2)
    assert float(one.norm()) > 0 and float((out - one).norm()) <= 0.016 * float(one.norm())


def test_kv_read_without_sequences():
    """All rows are padding then, and padding reads as zeros."""
    cache = mx.KVCache(2, 16, 1, 64)
    ko, vo = (torch.full((5, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens, starts = torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = mx.alloc_workspace(256)
    mx.mx_kv_read(cache, none, lens, starts, ko, vo, ws)
    assert mx.moe_get_status(ws) == 0
    assert float(ko.abs().sum()) == 0 and float(vo.abs().sum()) == 0
