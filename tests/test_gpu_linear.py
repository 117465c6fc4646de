"""GPU parity of the MX projections (mx_linear) against fp64 products of the decoded operands."""
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


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _weights(N, K, fmt, seed):
    """Codes and scales on the GPU, of weights whose rows and blocks differ in size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(N, K, generator=g, device="cuda") * torch.exp(torch.randn(N, K // 32, generator=g, device="cuda")).repeat_interleave(32, 1)
    codes = torch.empty(N, K // (2 if fmt == "e2m1" else 1), dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")
    mx.mx_quantize_weights(w, fmt, codes, scales)
    return codes, scales


def _values(codes, scales, fmt):
    """fp64 on the GPU."""
    table = ref.E4M3.cuda() if fmt == "e4m3" else torch.cat((ref.E2M1, -ref.E2M1)).cuda()
    c = codes.long() if fmt == "e4m3" else torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return (table[c].unflatten(-1, (-1, 32)) * torch.exp2(scales.double() - 127).unsqueeze(-1)).flatten(-2)


def _run(T, N, K, w_fmt, act, out, bias=False, seed=0, given=False, ws=None):
    codes, scales = _weights(N, K, w_fmt, seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, K, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))).to(torch.bfloat16)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    xc = torch.empty(T, K // (2 if act == "e2m1" else 1), dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, K // 32, dtype=torch.uint8, device="cuda")
    mx.mx_quantize_act(x, xc, xs, fmt=act)
    w = mx.LinearWeights(codes, scales, w_fmt)
    got = torch.full((T, N), float("nan"), dtype=DT[out], device="cuda")
    ws = mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, K, act)) if ws is None else ws
    if given:
        mx.mx_linear(w, got, ws, codes=xc, scales=xs, act_fmt=act, bias=b)
    else:
        mx.mx_linear(w, got, ws, x=x, act_fmt=act, bias=b)
    assert mx.moe_get_status(ws) == 0
    a, v = _values(xc, xs, act), _values(codes, scales, w_fmt)
    want, size = a @ v.T, a.abs() @ v.abs().T
    if bias:
        want, size = want + b.double(), size + b.double().abs()
    # products of K = 32 are added to the sum one after the other, each aligned to the larger
    # and cut to fp32 (2^-23 a time), within a product the same over some parts of it; the
    # parts of a split K and the bias beside
    tol = torch.finfo(DT[out]).eps / 2 * want.abs() + (K / 32 + 32) * 2.0 ** -23 * size
    assert torch.all((got.double() - want).abs() <= tol), float(((got.double() - want).abs() / tol).max())
    # the rounding apart, sums are far better than that bound on the whole
    if out == "f32":
        assert float((got.double() - want).norm() / want.norm()) < 1e-5
    return got


FORMATS = [("e4m3", "e4m3"), ("e2m1", "e4m3"), ("e2m1", "e2m1")]


@pytest.mark.parametrize("w_fmt,act", FORMATS)
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 128, 128), (3, 129, 96), (16, 256, 512), (17, 300, 1056), (64, 1000, 4096), (100, 384, 2080),
                                   (129, 257, 160), (256, 130, 640), (5, 6144, 4096), (200, 513, 8192)])
def test_few_tokens(T, N, K, w_fmt, act):
    _run(T, N, K, w_fmt, act, "f32", seed=T + N)
    _run(T, N, K, w_fmt, act, "bf16", bias=True, seed=T + N + 1, given=True)


@pytest.mark.parametrize("w_fmt,act", FORMATS)
@pytest.mark.parametrize("T,N,K", [(257, 256, 256), (300, 128, 32), (384, 100, 96), (385, 641, 1056), (1000, 1537, 416), (2049, 2048, 1024), (700, 33, 8192)])
def test_many_tokens(T, N, K, w_fmt, act):
    _run(T, N, K, w_fmt, act, "f32", seed=T + N)
    _run(T, N, K, w_fmt, act, "bf16", bias=True, seed=T + N + 1, given=True)


@pytest.mark.parametrize("w_fmt,act", FORMATS)
def test_more_tiles_than_a_gpu_holds(w_fmt, act):
    """Each CTA goes through several tiles: a vocabulary for few tokens, a prompt for many."""
    _run(20, 40003, 512, w_fmt, act, "bf16", seed=1)
    _run(250, 40002, 256, w_fmt, act, "bf16", seed=2)
    _run(5000, 3000, 512, w_fmt, act, "bf16", seed=3)
    _run(3001, 5001, 160, w_fmt, act, "f32", seed=4)


def test_given_codes_and_a_used_workspace_change_nothing():
    """bf16 activations and their own codes give the same bits, on a workspace that larger
    and smaller calls have used, and in a call after another."""
    ws = mx.alloc_workspace(mx.mx_linear_workspace_size(2100, 640, 1056, "e4m3"))
    for T in (2100, 5, 300, 128, 1, 257, 64):
        for w_fmt, act in FORMATS:
            a = _run(T, 640, 1056, w_fmt, act, "bf16", seed=9, ws=ws)
            b = _run(T, 640, 1056, w_fmt, act, "bf16", seed=9, given=True)
            assert torch.equal(a, b)


def test_rows_do_not_depend_on_the_others():
    """A token whose activations are NaN or huge leaves the other rows of its tile alone."""
    N, K = 300, 1056
    codes, scales = _weights(N, K, "e2m1", 3)
    w = mx.LinearWeights(codes, scales, "e2m1")
    for T in (40, 600):
        x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
        out, ws = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)], mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, K))
        mx.mx_linear(w, out[0], ws, x=x)
        x[7] = float("nan")
        x[T - 2] = 1e38
        mx.mx_linear(w, out[1], ws, x=x)
        rest = [t for t in range(T) if t not in (7, T - 2)]
        assert torch.equal(out[0][rest], out[1][rest]) and not torch.equal(out[0][T - 2], out[1][T - 2])


def test_zero_rows_and_the_largest_values():
    N, K, T = 256, 256, 9
    w = torch.full((N, K), 448.0, device="cuda")
    codes, scales = torch.empty(N, K, dtype=torch.uint8, device="cuda"), torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")
    mx.mx_quantize_weights(w, "e4m3", codes, scales)
    x = torch.zeros(T, K, device="cuda")
    x[3], x[5], x[6] = 1.0, -2.0 ** 100, 2.0 ** -130
    out, ws = torch.empty(T, N, device="cuda"), mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, K))
    mx.mx_linear(mx.LinearWeights(codes, scales, "e4m3"), out, ws, x=x.to(torch.bfloat16))
    assert torch.all(out[[0, 1, 2, 4, 7, 8]] == 0)
    assert torch.all(out[3] == 448.0 * K) and torch.all(out[5] == -448.0 * K * 2.0 ** 100)
    assert torch.all((out[6] - 448.0 * K * 2.0 ** -130).abs() <= 448.0 * K * 2.0 ** -130 * 2.0 ** -4)


def test_two_streams_and_a_graph():
    N, K = 640, 1024
    weights = [mx.LinearWeights(*_weights(N, K, f, i), f) for i, f in enumerate(("e4m3", "e2m1"))]
    xs = [torch.randn(T, K, device="cuda").to(torch.bfloat16) for T in (33, 700)]
    ws = [mx.alloc_workspace(mx.mx_linear_workspace_size(700, N, K)) for _ in range(3)]
    want = [torch.empty(x.shape[0], N, device="cuda") for x in xs]
    for w, x, o in zip(weights, xs, want):
        mx.mx_linear(w, o, ws[0], x=x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[torch.empty_like(o) for o in want] for _ in range(6)]
    for outs in got:
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                mx.mx_linear(weights[i], outs[i], ws[1 + i], x=xs[i])
    torch.cuda.synchronize()
    graph, last = torch.cuda.CUDAGraph(), [torch.empty_like(o) for o in want]
    with torch.cuda.graph(graph):
        for w, x, o in zip(weights, xs, last):
            mx.mx_linear(w, o, ws[0], x=x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for outs in got + [last]:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_wait_that_runs_out_is_reported():
    """A limit of a nanosecond: waits end, the status says so, and the next call is whole."""
    for T, N in ((8, 2048), (8, 40000), (1000, 2048)):   # K shared by a cluster, whole, pairs
        codes, scales = _weights(N, 4096, "e4m3", 1)
        w = mx.LinearWeights(codes, scales, "e4m3")
        x, ws = torch.randn(T, 4096, device="cuda").to(torch.bfloat16), mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, 4096))
        out, again = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
        mx.mx_linear(w, out, ws, x=x)
        mx.mx_debug_set_wait_limit_ns(1)
        try:
            mx.mx_linear(w, again, ws, x=x)
            assert mx.moe_get_status(ws) == mx.MX_ERR_TIMEOUT
        finally:
            mx.mx_debug_set_wait_limit_ns(2000000000)
        mx.mx_linear(w, again, ws, x=x)
        assert mx.moe_get_status(ws) == 0 and torch.equal(out, again)


@pytest.mark.parametrize("T,N,wf,af", [(700, 6144, "e4m3", "e4m3"), (300, 2000, "e2m1", "e2m1"), (65, 30000, "e2m1", "e4m3")])
def test_pairs_leave_together_where_waits_run_out(T, N, wf, af):
    """In a pair either CTA's wait may be the one that runs out, at any point of the other's
    way: limits from one that ends all waits to one that ends few, and whole calls between."""
    K = 2048
    w = mx.LinearWeights(*_weights(N, K, wf, 3), wf)
    x, ws = torch.randn(T, K, device="cuda").to(torch.bfloat16), mx.alloc_workspace(mx.mx_linear_workspace_size(T, N, K, af))
    out, again = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    mx.mx_linear(w, out, ws, x=x, act_fmt=af)
    assert mx.moe_get_status(ws) == 0
    for limit in (1, 1000, 4000, 12000):
        mx.mx_debug_set_wait_limit_ns(limit)
        try:
            for _ in range(2):
                mx.mx_linear(w, again, ws, x=x, act_fmt=af)
            assert mx.moe_get_status(ws) in (0, mx.MX_ERR_TIMEOUT)
        finally:
            mx.mx_debug_set_wait_limit_ns(2000000000)
        mx.mx_linear(w, again, ws, x=x, act_fmt=af)
        assert mx.moe_get_status(ws) == 0 and torch.equal(out, again)
