"""The operators of a decoding step together: a block with MX projections, positions and
sandwich norms over a ragged batch, each stage against its reference given what the stage
before it left, and tokens drawn from its output."""
import pytest
import torch

from block_scaled_mx_gb300 import block as B
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


H, I, E, K, HQ, HK, D, PAGE = 256, 128, 8, 2, 8, 2, 64, 16


def _sandwich(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return B.Sandwich(post=(1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16),
                      gate=torch.randn(H, generator=g, device="cuda").to(torch.bfloat16), gate_act="sigmoid", block_scale=1.5, residual_scale=0.875)


def _block(**kw):
    return B.random_block(H, I, E, K, HQ, HK, D, seed=3, projections="e2m1", rope=mx.Rope(D, layout="half"), before=_sandwich(1),
                          between=_sandwich(2), **kw)


def test_block_stages(monkeypatch):
    """Each call of a forward pass, recorded with what it was given, against its definition."""
    calls = []

    def record(name):
        f = getattr(mx, name)

        def wrapped(*a, **kw):
            a0 = [t.clone() if isinstance(t, torch.Tensor) else t for t in a]
            kw0 = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}
            f(*a, **kw)
            calls.append((name, a0, kw0, a, kw))

        monkeypatch.setattr(mx, name, wrapped)

    blk = _block()
    for name in ("mx_sandwich_rmsnorm", "mx_linear", "mx_rope_kv_append", "mx_paged_attention"):
        record(name)
    g = torch.Generator(device="cuda").manual_seed(4)
    full = ref.make_batch([1, 1, 1], [90, 40, 20], PAGE, 5)
    cache = mx.KVCache(full.pages, PAGE, HK, D)
    kv = [0, 0, 0]
    for new in ([70, 1, 9], [1, 1, 1], [12, 1, 0]):
        kv = [a + b for a, b in zip(kv, new)]
        batch = ref.Batch(new, list(kv), PAGE, full.pages, full.table)
        x = torch.randn(batch.T, H, generator=g, device="cuda")
        res = torch.randn(batch.T, H, generator=g, device="cuda").to(torch.bfloat16)
        calls.clear()
        out, after = blk.forward(x, res, cache, *batch.device(), max(new))
        assert blk.status() == 0
        assert [c[0] for c in calls] == ["mx_sandwich_rmsnorm", "mx_linear", "mx_rope_kv_append", "mx_paged_attention", "mx_linear", "mx_sandwich_rmsnorm"]
        # the residual stream through both norms: each rounded to bf16, the norms' fp32 a few 2^-20 beside
        for (_, a0, kw0, a, kw), s in zip((calls[0], calls[5]), (blk.before, blk.between)):
            n = a0[0].double()
            n = n / torch.sqrt((n * n).mean(1, keepdim=True) + 1e-6) * s.post.double()
            z = 0.875 * a0[3].double() + 1.5 * torch.sigmoid(s.gate.double()) * n
            assert torch.all((a[4].double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -18 * (n.abs() + a0[3].double().abs()))
        assert torch.equal(calls[5][3][4], after)
        # the first projection: the norm's codes, decoded, times the weights' (as fp64 of what they stand for)
        a = ref.decode(calls[1][2]["codes"].cpu(), calls[1][2]["scales"].cpu(), "e4m3")
        w = _decoded_weights(3)[0]
        want, size = a @ w.T, a.abs() @ w.abs().T
        qkv = calls[2][1]   # q, k, v before the rotation
        got = torch.cat([qkv[2].flatten(1), qkv[3].flatten(1), qkv[4].flatten(1)], 1).cpu().double()
        assert torch.all((got - want).abs() <= 2.0 ** -8 * want.abs() + (H / 32 + 32) * 2.0 ** -23 * size)
        # positions
        pos = torch.cat([torch.arange(b - n, b) for n, b in zip(batch.n, batch.kv)])
        f, amp = srv.frequencies(D)
        turned, size = srv.rotate(qkv[2].cpu().double(), pos, f, amp, D, "half")
        assert torch.all((blk.last["q"].cpu().double() - turned).abs() <= 2.0 ** -8 * turned.abs() + 2.0 ** -20 * size)
        # attention, from the rotated queries and what the cache holds
        tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        o, _, tol, _ = ref.attention(blk.last["q"].cpu(), *tables, "e4m3", batch, D ** -0.5, True, 0)
        assert torch.all((blk.last["att"].cpu().double() - o).abs() <= tol)


def _decoded_weights(seed):
    """The projections' weights of the block of this seed, as the values of their codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, fan_in):
        return torch.randn(*shape, generator=g, device="cuda") * fan_in ** -0.5

    for rows, cols in ((2 * I, H), (H, I)):
        for _ in range(E + 1):
            normal(rows, cols, fan_in=cols)
    out = []
    for rows, cols in (((HQ + 2 * HK) * D, H), (H, HQ * D)):
        w = normal(rows, cols, fan_in=cols)
        codes, scales = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
        mx.mx_quantize_weights(w, "e2m1", codes, scales)
        out.append(ref.decode(codes.cpu(), scales.cpu(), "e2m1"))
    return out


def test_tokens_follow_the_logits():
    V, n = 1003, 6
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(V, H, generator=g, device="cuda") * H ** -0.5
    x = torch.randn(n, H, generator=g, device="cuda")
    res = torch.randn(n, H, generator=g, device="cuda").to(torch.bfloat16)
    u = torch.rand(n, generator=g, device="cuda")
    rules = dict(temperature=torch.tensor([0.7, 1.0, 0.0, 1.3, 1.0, 2.0], device="cuda"), top_k=torch.tensor([50, 0, 9, 1, 300, 0], dtype=torch.int32, device="cuda"),
                 top_p=torch.tensor([0.9, 0.5, 0.9, 1.0, 0.99, 1.0], device="cuda"), min_p=torch.tensor([0.0, 0.01, 0.0, 0.0, 0.05, 0.1], device="cuda"))
    ones = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    for weights, before in ((w.to(torch.bfloat16), None), (B.random_weights(w, "e4m3"), _sandwich(5))):
        head = B.TokenHead(ones, weights, before=before)
        tokens, logp, logits = head.forward(x, res, u, **rules)
        assert head.status() == 0
        for t in range(n):
            want, lp, margin = srv.sample(logits[t].float().tolist(), float(u[t]), float(rules["temperature"][t]), int(rules["top_k"][t]), float(rules["top_p"][t]),
                                          float(rules["min_p"][t]))
            assert int(tokens[t]) == want or margin < 2.0 ** -29
            assert int(tokens[t]) != want or abs(float(logp[t]) - lp) <= 2.0 ** -20 * (1 + abs(lp))


def test_generation_in_pieces_is_generation_at_once():
    """A prompt in one step, or in chunks: the cache holds the same codes up to the rounding
    of a step's projections, which do not depend on the step's size."""
    blk = _block(keep_last=False)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(100, H, generator=g, device="cuda")
    res = torch.randn(100, H, generator=g, device="cuda").to(torch.bfloat16)
    full = ref.make_batch([1], [100], PAGE, 5)
    caches = [mx.KVCache(full.pages, PAGE, HK, D) for _ in range(2)]
    blk.forward(x, res, caches[0], *ref.Batch([100], [100], PAGE, full.pages, full.table).device(), 100)
    at = 0
    for n in (33, 1, 60, 6):
        blk.forward(x[at:at + n], res[at:at + n], caches[1], *ref.Batch([n], [at + n], PAGE, full.pages, full.table).device(), n)
        at += n
    assert blk.status() == 0
    # sums of a split or a whole K differ by (H / 32 + 32) 2^-23 of their terms' sizes and are
    # rounded to bf16 (2^-8), then to a code (2^-4): at most a step of 2^-3 where they differ
    a, b = (ref.decode(c.k_codes.cpu(), c.k_scales.cpu(), "e4m3") for c in caches)
    low = 2.0 ** -9 * torch.exp2(torch.maximum(caches[0].k_scales, caches[1].k_scales).cpu().double() - 127).repeat_interleave(32, -1)
    assert torch.all((a - b).abs() <= 2.0 ** -3 * torch.maximum(a.abs(), b.abs()) + low)


def test_block_with_mx_projections_in_a_graph():
    """A decoding step captured once and replayed for the next tokens."""
    blk = _block(keep_last=False)
    ones = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    head = B.TokenHead(ones, B.random_weights(torch.randn(503, H, device="cuda"), "e2m1"), before=_sandwich(4))
    full = ref.make_batch([1] * 3, [40, 9, 21], PAGE, 5)
    cache = mx.KVCache(full.pages, PAGE, HK, D)
    table = full.table.cuda()
    lens, starts = torch.tensor([30, 2, 20], dtype=torch.int32, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    x, u = torch.randn(3, H, device="cuda"), torch.rand(3, device="cuda")
    res = torch.randn(3, H, device="cuda").to(torch.bfloat16)

    def step():
        out, after = blk.forward(x, res, cache, table, lens, starts, 1)
        return head.forward(out, after, u, top_k=torch.full((3,), 20, dtype=torch.int32, device="cuda"))

    want = []
    for _ in range(2):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, logp, logits = step()
    for i in range(3):
        x.copy_(torch.randn(3, H, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
        u.fill_(0.2 + 0.3 * i)
        graph.replay()
        torch.cuda.synchronize()
        for t in range(3):
            got, _, margin = srv.sample(logits[t].tolist(), float(u[t]), top_k=20)
            assert int(tokens[t]) == got or margin < 2.0 ** -29
        want.append(tokens.tolist())
        lens += 1
    assert blk.status() == 0 and head.status() == 0


def test_main_generates(capsys):
    B.main(prompts=(40, 3), steps=2, H=256, I=128, E=4, k=2, n_heads=4, n_kv_heads=1, head_dim=64, page=16, vocabulary=515)
    out = capsys.readouterr().out
    assert "step 2" in out and "next" in out
