"""GPU parity of sampling (mx_sample) against a sort in 64 bits."""
import math

import pytest
import torch

from block_scaled_mx_gb300 import mxmoe as mx

import serve_reference as srv

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as g

    g.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _draw(logits, u, status=0, **rules):
    """Tokens and log-probabilities of logits (a CUDA tensor) under per-row lists."""
    T, V = logits.shape
    kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
    kw = {n: torch.tensor(v, dtype=kinds[n], device="cuda") for n, v in rules.items()}
    tokens = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((T,), 7.0, device="cuda")
    ws = mx.alloc_workspace(mx.mx_sample_workspace_size(T, V))
    mx.mx_sample(logits, torch.tensor(u, dtype=torch.float32, device="cuda"), tokens, ws, logp=logp, **kw)
    assert mx.moe_get_status(ws) == status
    return tokens.tolist(), logp.tolist()


def _check(logits, u, **rules):
    got, logp = _draw(logits, u, **rules)
    rows = logits.float().cpu().tolist()
    for t, row in enumerate(rows):
        # what the call reads: fp32 numbers
        one = {n: float(torch.tensor(v[t], dtype=torch.float32)) if n != "top_k" else v[t] for n, v in rules.items()}
        want, lp, margin = srv.sample(row, float(torch.tensor(u[t], dtype=torch.float32)), **one)
        # weights are 2^-30 off: a draw as near as that to a border may go to either side
        assert got[t] == want or margin < 2.0 ** -29, (t, got[t], want, margin)
        if got[t] == want:
            # the logit's difference and product in fp32 (2^-23 of it), two logarithms (2^-22 of
            # values below 20), for a token of few units of 2^-43 their rounding (2^-13 of those that are drawn)
            assert abs(logp[t] - lp) <= 2.0 ** -20 * (1 + abs(lp)), (t, logp[t], lp)


def _random(T, V, dtype, seed, spread=2.5, stride=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V + stride, generator=g) * spread
    x[torch.rand(T, V + stride, generator=g) < 0.02] = -INF
    return x.to(dtype).cuda()[:, :V], [float(v) for v in torch.rand(T, generator=g)]


RULES = [dict(), dict(temperature=0.7), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=1.5, top_k=300, top_p=0.8, min_p=0.01),
         dict(temperature=0.0), dict(top_k=1), dict(temperature=0.05, top_k=1000), dict(top_p=0.999, temperature=2.0), dict(top_k=10 ** 6, top_p=1.0),
         dict(temperature=30.0, top_p=0.5), dict(temperature=0.01, top_k=700, top_p=0.9999)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 20011])
def test_rules(V, dtype):
    for i, rules in enumerate(RULES):
        T = 5
        logits, u = _random(T, V, dtype, 100 * V + i)
        if V <= 2:
            logits = torch.where(torch.isinf(logits), torch.zeros_like(logits), logits)
        _check(logits, u, **{n: [v] * T for n, v in rules.items()})


@pytest.mark.parametrize("dtype,V", [(torch.float32, 100003), (torch.bfloat16, 131072), (torch.bfloat16, 151937)])
def test_large_vocabularies_with_rules_of_their_own(V, dtype):
    T = 13
    logits, u = _random(T, V, dtype, V, 2.0, stride=5)     # rows start anywhere
    _check(logits, u, **{n: [RULES[t].get(n, d) for t in range(T)] for n, d in dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0).items()})


def test_the_largest_vocabularies():
    for dtype, V in ((torch.float32, 400000), (torch.bfloat16, 800000)):
        x = torch.full((2, V), -3.0, dtype=dtype, device="cuda")
        x[0, V - 1] = 20.0
        x[1, 0] = 20.0
        assert _draw(x, [0.5, 0.999], top_p=[0.5, 0.5])[0] == [V - 1, 0]
        # all of one logit but one: e^-23 V of the weight is the others'
        tokens, _ = _draw(x, [0.5, 0.0], top_k=[V - 1, V - 1])
        assert tokens == [V - 1, 0]
    with pytest.raises(mx.MxError):
        _draw(torch.zeros(1, 400001, device="cuda"), [0.5])


@pytest.mark.parametrize("V", [7, 600, 5000, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits(V, dtype):
    """Ties go by number: the first k, or the first whose weights reach p."""
    T = 6
    x = torch.full((T, V), 1.25, dtype=dtype, device="cuda")
    x[3, V // 2] = 1.0
    u = [0.0, 0.37, 1 - 2.0 ** -24, 0.9, 0.5, 0.25]
    for rules in (dict(), dict(top_k=[V // 2 + 1] * T), dict(top_p=[0.3] * T), dict(top_k=[V - 1] * T, top_p=[0.61] * T), dict(min_p=[1.0] * T),
                  dict(min_p=[7.0] * T), dict(temperature=[0.0] * T)):
        if rules.get("min_p", [0])[0] > 1:
            assert _draw(x, u, **rules)[0] == _draw(x, u, min_p=[1.0] * T)[0]
        else:
            _check(x, u, **rules)


def test_many_logits_in_one_bin():
    """Logits so near each other that the histogram's bin holds thousands: the bits decide."""
    g = torch.Generator().manual_seed(3)
    for V, scale, T in ((20000, 1e-3, 4), (20000, 1e-7, 4), (5000, 1e-30, 4)):
        x = torch.randn(T, V, generator=g) * scale
        x[1] += 5.0                       # a grid of 2^-22 about 5: many are equal
        x[2] = x[2].abs() * -1
        x[2, ::2] = 0.0
        x[2, 1::4] = -0.0                 # both zeros are the same logit
        x[3] = (x[3] / scale).to(torch.bfloat16).float() * 1e-2
        u = [float(v) for v in torch.rand(T, generator=g)]
        for rules in (dict(top_k=[3000] * T), dict(top_p=[0.4] * T), dict(top_k=[1500, 2500, 4000, 600], top_p=[0.77] * T)):
            _check(x.cuda(), u, **rules)


def test_masks():
    """Rows that are banned but for a few, by -inf and by the type's lowest value; far logits below."""
    V = 3001
    g = torch.Generator().manual_seed(4)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.full((8, V), -INF)
        x[0, 17] = -5.0                                   # the only one left
        x[1, [3, 2999]] = torch.tensor([1.0, 1.0])
        x[2] = torch.finfo(dtype).min
        x[2, 5:9] = torch.randn(4, generator=g)
        x[3] = torch.finfo(dtype).min                     # all of them banned alike: any may be drawn
        x[4] = torch.randn(V, generator=g) - 1e4
        x[4, :5] = 0.0
        x[5] = torch.randn(V, generator=g)
        x[5, 40] = x[5, 41] = INF                          # the only ones drawn
        x[6] = torch.randn(V, generator=g) * 1e30
        x[7] = torch.randn(V, generator=g) * 1e-38
        x = x.to(dtype)
        u = [0.5, 0.75, 0.4, 0.61, 0.1, 0.7, 0.3, 0.999]
        for rules in (dict(), dict(top_k=[50] * 8), dict(top_p=[0.7] * 8), dict(top_k=[5] * 8, top_p=[0.9] * 8, min_p=[0.2] * 8), dict(temperature=[0.0] * 8)):
            tokens, _ = _draw(x.cuda(), u, **rules)
            # two of half the weight each: top_p 0.7 keeps both
            assert tokens[5] == (40 if "temperature" in rules else 41)
            rows = [0, 1, 2, 3, 4, 6, 7]
            _check(x.cuda()[rows], [u[r] for r in rows], **{n: [v[r] for r in rows] for n, v in rules.items()})


def test_rows_without_an_answer():
    """NaN, nothing but -inf, a negative or NaN temperature: token -1, and the status says so;
    other rows are drawn."""
    V = 50
    x = torch.randn(6, V)
    x[0, 3] = math.nan
    x[1] = -INF
    good = x[4].tolist()
    tokens, logp = _draw(x.cuda(), [0.5] * 6, status=mx.MX_ERR_DEVICE_ARG, temperature=[1.0, 1.0, -1.0, math.nan, 1.0, INF])
    assert tokens[:4] == [-1] * 4 and all(math.isnan(v) for v in logp[:4])
    assert tokens[4] == srv.sample(good, 0.5)[0]
    assert tokens[5] == 25      # an infinite temperature: all alike


def test_random_numbers_at_the_ends():
    x = torch.randn(4, 999, generator=torch.Generator().manual_seed(1)).cuda()
    lo, hi = _draw(x, [0.0] * 4)[0], _draw(x, [1 - 2.0 ** -24] * 4)[0]
    assert lo == [0] * 4 and hi == [998] * 4
    assert _draw(x, [-3.0] * 4)[0] == lo and _draw(x, [1.0] * 4)[0] == hi and _draw(x, [math.nan] * 4)[0] == lo


def test_frequencies_follow_the_probabilities():
    """4096 equally spaced random numbers: each token is drawn as often as its share, to one."""
    x = torch.tensor([[0.0, 1.0, -INF, 2.0, -1.0, 0.5]])
    n = 4096
    tokens, _ = _draw(x.expand(n, 6).contiguous().cuda(), [(i + 0.5) / n for i in range(n)])
    p = torch.softmax(x[0].double(), 0)
    for i in range(6):
        assert abs(tokens.count(i) - n * float(p[i])) <= 1


def test_the_same_call_again_on_another_stream_and_in_a_graph():
    T, V = 40, 60001
    logits, u = _random(T, V, torch.float32, 77)
    u = torch.tensor(u, device="cuda")
    kw = dict(top_k=torch.full((T,), 200, dtype=torch.int32, device="cuda"), top_p=torch.full((T,), 0.9, device="cuda"))
    outs = [(torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")) for _ in range(3)]
    ws = [mx.alloc_workspace(256) for _ in range(3)]
    mx.mx_sample(logits, u, outs[0][0], ws[0], logp=outs[0][1], **kw)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        mx.mx_sample(logits, u, outs[1][0], ws[1], logp=outs[1][1], **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_sample(logits, u, outs[2][0], ws[2], logp=outs[2][1], **kw)
    graph.replay()
    torch.cuda.synchronize()
    for tokens, logp in outs[1:]:
        assert torch.equal(tokens, outs[0][0]) and torch.equal(logp, outs[0][1])


def _groups(V, groups, rest, T, dtype, seed):
    """T rows of (count, logit) groups in shuffled places, the others at `rest`."""
    x = torch.full((T, V), rest)
    for t in range(T):
        places, at = torch.randperm(V, generator=torch.Generator().manual_seed(seed + t)), 0
        for n, v in groups:
            x[t, places[at:at + n]] = v
            at += n
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,groups,rest,rules", [
    (5000, [(1000, 1.0), (200, 1 - 1 / 128), (100, 1 - 2 / 128)], -20.0, dict(top_p=0.87)),
    (5000, [(1, 0.0), (1000, -1 / 128), (1000, -2 / 128)], -100.0, dict(top_p=0.3)),
    (40000, [(1000, 1.0), (260, 1 - 1 / 128), (100, 1 - 2 / 128)], -20.0, dict(top_k=1250)),
    (40000, [(1000, 1.0), (260, 1 - 1 / 128), (100, 1 - 2 / 128)], -20.0, dict(top_k=1250, top_p=0.93)),
    (2000, [(900, 1.0), (300, 1 - 1 / 128), (700, 1 - 2 / 128)], -1.0, dict(top_k=1100)),
])
def test_prefixes_that_end_at_a_border_with_many_neighbours(V, groups, rest, rules, dtype):
    """At this temperature the histogram's bins are 1/128 wide and these logits lie on their
    borders: up to the prefix's end there are fewer tokens than a CTA's list holds (1280),
    with those on the border more."""
    T = 8
    _check(_groups(V, groups, rest, T, dtype, V), [(t + 0.5) / T for t in range(T)], temperature=[0.25] * T, **{n: [v] * T for n, v in rules.items()})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_k_and_top_p_that_end_among_thousands_of_equal_logits(dtype):
    """Both ends lie among equal logits, whose last bits the search never needs: two
    selections one right behind the other, in the same bin or in two."""
    V, T = 30011, 12
    x = torch.randint(0, 3, (T, V), generator=torch.Generator().manual_seed(6)) * 0.5
    u = [(t + 0.5) / T for t in range(T)]
    x = x.to(dtype).cuda()
    for rules in (dict(top_k=[25000] * T, top_p=[0.8] * T), dict(top_k=[9000 + 1700 * t for t in range(T)], top_p=[0.4 + 0.05 * t for t in range(T)])):
        want = None
        for _ in range(5):
            if want is None:
                _check(x, u, **rules)
                want = _draw(x, u, **rules)
            assert _draw(x, u, **rules) == want


@pytest.mark.parametrize("V,dtype", [(4100, torch.float32), (9001, torch.float32), (131072, torch.bfloat16)])
def test_clusters_that_start_beside_other_work(V, dtype):
    """Rows shared by two, four and eight CTAs, whose clusters start as another stream's leave:
    a CTA tells its peers a maximum only once they run."""
    T = 70
    logits, u = _random(T, V, dtype, V)
    rules = dict(temperature=[0.8] * T, top_k=[0, 40] * (T // 2), top_p=[0.9] * T)
    want = _draw(logits, u, **rules)
    kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32)
    kw = {n: torch.tensor(v, dtype=kinds[n], device="cuda") for n, v in rules.items()}
    u = torch.tensor(u, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[(torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")) for _ in range(30)] for _ in streams]
    ws = [mx.alloc_workspace(256) for _ in streams]
    torch.cuda.synchronize()
    for i in range(30):
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                mx.mx_sample(logits, u, o[i][0], w, logp=o[i][1], **kw)
    torch.cuda.synchronize()
    assert all((tokens.tolist(), logp.tolist()) == want for o in outs for tokens, logp in o) and not any(mx.moe_get_status(w) for w in ws)


@pytest.mark.parametrize("rules", [dict(), dict(top_p=0.9), dict(top_k=40), dict(top_k=1200, top_p=0.5), dict(min_p=0.1)])
def test_the_smallest_temperatures(rules):
    """Positive temperatures down to the smallest number; below 2^-126 they count as that."""
    V, temperature = 1009, [2.0 ** -149, 1e-40, 4.1e-39, 2.0 ** -126, 1e-37, 1e-30]
    T = len(temperature)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(T, V, generator=torch.Generator().manual_seed(11)).to(dtype)
        x[:, 500] = x[:, 7] = 6.0                      # the two largest share the draw
        kw = {n: [v] * T for n, v in rules.items()}
        for u, place in ((0.25, 7), (0.75, 500)):
            tokens, logp = _draw(x.cuda(), [u] * T, temperature=temperature, **kw)
            alone = rules.get("top_p", 1.0) <= 0.5     # the first of the two has half of the weight
            assert tokens == [7 if alone else place] * T
            assert all(abs(v - (0.0 if alone else math.log(0.5))) <= 2.0 ** -23 for v in logp)
    x = torch.full((4, V), -1.0)
    x[:, 3], x[:, 9] = 2.0 ** -126, 0.0                # one unit of 2^-126 apart: weights 1 and 1 / e
    tokens, logp = _draw(x.cuda(), [0.7, 0.75, 0.7, 0.75], temperature=[2.0 ** -126, 2.0 ** -126, 2.0 ** -140, 2.0 ** -140])
    share = 1 / (1 + math.exp(-1))                     # 0.731
    assert tokens == [3, 9, 3, 9]
    assert all(abs(v - w) <= 2.0 ** -20 * (1 + abs(w)) for v, w in zip(logp, [math.log(share), math.log(1 - share)] * 2))


@pytest.mark.parametrize("n", [2, 4, 9, 300, 3000])
def test_infinite_logits_share_the_draw(n):
    """n logits of +inf are alike: each is drawn with 1 / n, and the log-probability is a number."""
    V, T = 7001, 5
    x = torch.randn(T, V, generator=torch.Generator().manual_seed(n))
    places = torch.randperm(V, generator=torch.Generator().manual_seed(n))[:n].sort().values
    x[:, places] = INF
    u = [(t + 0.5) / T for t in range(T)]
    for rules, kept in ((dict(), n), (dict(top_k=[50] * T), min(n, 50)), (dict(top_p=[0.7] * T), math.ceil(float(torch.tensor(0.7)) * n)), (dict(min_p=[0.5] * T), n)):
        for dtype in (torch.float32, torch.bfloat16):
            tokens, logp = _draw(x.to(dtype).cuda(), u, **rules)
            # u as the call reads it: in fp32, where 0.7 and 0.9 lie below the borders 210 / 300 and 270 / 300
            assert tokens == [int(places[int(float(v) * kept)]) for v in torch.tensor(u, dtype=torch.float32)], rules
            # the logarithm of a whole number in fp32: its rounding and the function's, 2^-23 each
            assert all(abs(v + math.log(kept)) <= 2.0 ** -22 * math.log(kept) for v in logp), rules


def test_rules_that_are_not_numbers():
    """A NaN among a row's rules: no token, and the status says so; other rows are drawn."""
    x = torch.randn(4, 300, generator=torch.Generator().manual_seed(8)).cuda()
    fine = _draw(x, [0.3] * 4, top_p=[0.9] * 4, min_p=[0.01] * 4)
    for kw in (dict(top_p=[0.9, math.nan, 0.9, 0.9], min_p=[0.01] * 4), dict(top_p=[0.9] * 4, min_p=[0.01, math.nan, 0.01, 0.01])):
        tokens, logp = _draw(x, [0.3] * 4, status=mx.MX_ERR_DEVICE_ARG, **kw)
        assert tokens[1] == -1 and math.isnan(logp[1])
        assert [tokens[i] for i in (0, 2, 3)] == [fine[0][i] for i in (0, 2, 3)] and [logp[i] for i in (0, 2, 3)] == [fine[1][i] for i in (0, 2, 3)]
