"""GPU parity of mx_paged_attention against a plain fp64 reference: ragged
batches, head layouts, page sizes, windows, rows that see nothing, garbage in
places that no row sees, and refusals on the device."""
import math

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


def _setup(n, kv, heads, kv_heads, dim, page, fmt, seed=1, spread=0.5, garbage=True):
    """Batch, q (a strided slice) and a cache whose unused places hold NaN codes and scales."""
    batch = ref.make_batch(n, kv, page, seed)
    g = torch.Generator().manual_seed(seed + 100)
    q = torch.randn(max(batch.T, 1), heads * dim + 64, generator=g).to(torch.bfloat16)[: batch.T, : heads * dim]
    cache = mx.KVCache(batch.pages, page, kv_heads, dim, fmt)
    full = ref.Batch(list(kv), list(kv), page, batch.pages, batch.table)
    if full.T:
        k = torch.randn(full.T, kv_heads, dim, generator=g) * torch.exp(spread * torch.randn(1, kv_heads, dim, generator=g))
        v = torch.randn(full.T, kv_heads, dim, generator=g) * torch.exp(spread * torch.randn(full.T, kv_heads, 1, generator=g))
        if garbage:
            for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
                t.fill_(0x7F if t.shape[-1] > 4 else 0xFF)
        ws = mx.alloc_workspace(256)
        mx.mx_kv_append(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), *full.device(), ws)
        assert mx.moe_get_status(ws) == 0
    return batch, q.cuda().view(batch.T, heads, dim), cache


def _call(batch, q, cache, dev=None, **kw):
    T, heads, dim = q.shape
    out = torch.full((T, heads, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), 3.0, dtype=torch.float32, device="cuda")
    mq = kw.get("max_q_len", max(batch.n))
    ws = mx.alloc_workspace(mx.mx_paged_attention_workspace_size(T, len(batch.n), heads, cache.n_kv_heads, dim, mq))
    mx.mx_paged_attention(q, cache, *(dev or batch.device()), out, ws, lse=lse, **{"max_q_len": mq, **kw})
    return out, lse, mx.moe_get_status(ws), ws


def _compare(batch, q, cache, out, lse, fmt, scale, causal, window):
    tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    o, l, tol, tol_l = ref.attention(q.cpu(), *tables, fmt, batch, scale, causal, window)
    got, got_l = out.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isinf(got_l), torch.isinf(l))
    assert torch.all(torch.isfinite(got))
    bad = (got - o).abs() - tol
    assert float(bad.max()) <= 0, f"out: worst {float(bad.max())} over its bound at {bad.argmax()}"
    seen = ~torch.isinf(l)
    assert torch.all((got_l - l).abs()[seen] <= tol_l[seen])
    assert torch.all(got[~seen] == 0)


def _check(n, kv, heads, kv_heads, dim, page, fmt="e4m3", causal=True, window=0, scale=None, **kw):
    batch, q, cache = _setup(n, kv, heads, kv_heads, dim, page, fmt, **kw)
    out, lse, status, _ = _call(batch, q, cache, causal=causal, window=window, scale=scale)
    assert status == 0
    _compare(batch, q, cache, out, lse, fmt, dim ** -0.5 if scale is None else scale, causal, window)


SHAPES = [
    # one token, one key; one token, many
    ([1], [1], 1, 1, 64, 16), ([1], [1], 8, 1, 128, 64), ([1, 1, 1], [17, 64, 65], 8, 2, 128, 16),
    ([1], [700], 16, 1, 128, 128), ([1] * 5, [300, 1, 64, 33, 129], 13, 1, 64, 32),
    # drafts; a batch that mixes lengths, with an empty sequence and an empty cache
    ([6], [70], 16, 2, 128, 64), ([2, 0, 5, 1], [2, 0, 90, 200], 4, 4, 64, 48),
    # chunks
    ([40], [40], 8, 2, 128, 16), ([100, 1, 37], [150, 30, 37], 10, 2, 64, 16), ([65], [300], 5, 1, 128, 64),
    ([130, 3], [131, 259], 6, 3, 128, 32),
]


@pytest.mark.parametrize("n,kv,heads,kv_heads,dim,page", SHAPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_causal(n, kv, heads, kv_heads, dim, page, fmt):
    _check(n, kv, heads, kv_heads, dim, page, fmt)


@pytest.mark.parametrize("n,kv,heads,kv_heads,dim,page", SHAPES[2:])
def test_all_keys(n, kv, heads, kv_heads, dim, page):
    _check(n, kv, heads, kv_heads, dim, page, causal=False, seed=4)


@pytest.mark.parametrize("window", [1, 7, 64, 65, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("n,kv,heads,kv_heads,dim,page", [([1, 1], [300, 5], 8, 1, 128, 16), ([50, 3], [200, 100], 4, 2, 64, 32),
                                                          ([140], [400], 8, 8, 128, 64)])
def test_window(n, kv, heads, kv_heads, dim, page, window):
    _check(n, kv, heads, kv_heads, dim, page, window=window, seed=6)


def test_rows_that_see_nothing():
    """More new tokens than keys: the first ones' rows see no key; a sequence
    without keys; rows are zero with lse -inf, never NaN."""
    _check([5, 1, 20, 64], [2, 0, 0, 30], 8, 2, 128, 16)
    _check([5, 1, 20], [2, 0, 0], 8, 2, 64, 16, causal=False)


def test_long_split_segments():
    """Long contexts of few heads: every segment is split over many CTAs."""
    _check([1, 2], [20000, 3001], 2, 1, 128, 64, seed=8)
    _check([1], [9000], 8, 1, 64, 16, fmt="e2m1", seed=9)
    _check([9], [6000], 8, 1, 128, 32, seed=10)


def test_scale_and_peaked_scores():
    """Large scores: one key takes nearly all of a row's weight."""
    _check([3, 40], [80, 100], 4, 2, 128, 16, scale=4.0, seed=12)


@pytest.mark.parametrize("n,kv", [([1, 3], [200, 150]), ([70], [260])])
def test_values_of_far_apart_sizes(n, kv):
    """Tokens whose keys and values differ by 2^60, later (masked) ones among
    them: a row's result depends on what it sees alone."""
    heads, kv_heads, dim, page = 8, 2, 128, 16
    batch = ref.make_batch(n, kv, page, 21)
    g = torch.Generator().manual_seed(22)
    full = ref.Batch(list(kv), list(kv), page, batch.pages, batch.table)
    k = torch.randn(full.T, kv_heads, dim, generator=g)
    v = torch.randn(full.T, kv_heads, dim, generator=g) * torch.pow(2.0, torch.randint(-30, 31, (full.T, kv_heads, 1), generator=g).float())
    last = torch.tensor(full.starts[1:]) - 1
    v[last] *= 2.0 ** 40        # the newest token: only its own row sees it
    k[last] *= 2.0 ** 20
    q = torch.randn(batch.T, heads, dim, generator=g).to(torch.bfloat16)
    q[torch.tensor(batch.starts[1:]) - 1] *= 2.0 ** -20   # whose scores stay ordinary
    for fmt in ("e4m3", "e2m1"):
        cache = mx.KVCache(batch.pages, page, kv_heads, dim, fmt)
        ws = mx.alloc_workspace(256)
        mx.mx_kv_append(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), *full.device(), ws)
        out, lse, status, _ = _call(batch, q.cuda(), cache)
        assert status == 0
        _compare(batch, q.cuda(), cache, out, lse, fmt, dim ** -0.5, True, 0)


def test_pages_behind_the_window_may_be_gone():
    batch, q, cache = _setup([1, 20], [500, 400], 8, 2, 128, 16, "e4m3", seed=31)
    window = 50
    want, want_l, status, _ = _call(batch, q, cache, window=window)
    assert status == 0
    table, kv, starts = batch.device()
    table = table.clone()
    table[0, : (500 - window) // 16] = -1
    table[1, : (400 - 20 - window) // 16] = 2 ** 30
    out, lse, status, _ = _call(batch, q, cache, dev=(table, kv, starts), window=window)
    assert status == 0
    assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_bad_metadata_is_reported():
    """A bad page's keys are left out; a bad length or more new tokens than
    max_q_len leave the sequence's rows unwritten; padding rows too."""
    batch, q, cache = _setup([1, 2, 1, 4], [64, 40, 33, 50], 8, 2, 128, 16, "e4m3", seed=41)
    pad = torch.cat([q, q[:2]]).contiguous()
    table, kv, starts = (t.clone() for t in batch.device())
    table[0, 2] = -7            # keys 32 .. 47 of sequence 0
    kv[2] = 10 ** 9
    out, lse, status, ws = _call(batch, pad, cache, dev=(table, kv, starts), max_q_len=2)
    assert status == mx.MX_ERR_DEVICE_ARG
    assert mx.moe_get_status(ws) == 0
    assert torch.all(out[3:] == 3.0) and torch.all(lse[3:] == 3.0)
    # sequence 0 without the page's keys, from a batch that has only the others
    less = ref.Batch([1], [48], 16, batch.pages, torch.cat([batch.table[:1, :2], batch.table[:1, 3:4]], 1))
    tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    o, l, tol, tol_l = ref.attention(q[:1].cpu(), *tables, "e4m3", less, 128 ** -0.5, True, 0)
    assert torch.all((out[:1].cpu().double() - o).abs() <= tol) and torch.all((lse[:1].cpu().double() - l).abs() <= tol_l)


@pytest.mark.parametrize("n,kv", [([1] * 9, [900] * 9), ([90, 30], [700, 333])])
def test_same_bits_again_and_on_another_stream_and_in_a_graph(n, kv):
    batch, q, cache = _setup(n, kv, 8, 2, 128, 16, "e4m3", seed=51)
    want, want_l, status, ws = _call(batch, q, cache)
    assert status == 0
    dev = batch.device()
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            mx.mx_paged_attention(q, cache, *dev, out, ws, max_q_len=max(n), lse=lse)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_paged_attention(q, cache, *dev, out, ws, max_q_len=max(n), lse=lse)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    assert mx.moe_get_status(ws) == 0


def test_many_sequences():
    """More sequences than a block has threads."""
    n = [b % 3 for b in range(300)]
    kv = [t + (7 * b) % 50 for b, t in enumerate(n)]
    _check(n, kv, 4, 2, 64, 16, seed=61)


def test_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The chunk kernel's waits are bounded; a limit of zero makes them run out,
    which is reported and leaves the workspace ready."""
    n, kv = [90, 300], [700, 333]
    batch, q, cache = _setup(n, kv, 8, 2, 128, 16, "e4m3", seed=71)
    want, want_l, status, ws = _call(batch, q, cache)
    assert status == 0
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    try:
        mx.mx_debug_set_wait_limit_ns(0)
        mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
        assert mx.moe_get_status(ws) == mx.MX_ERR_TIMEOUT
    finally:
        mx.mx_debug_set_wait_limit_ns(2_000_000_000)
    mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
    assert mx.moe_get_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_few_rows_wait_that_runs_out():
    n, kv = [1] * 9, [900] * 9
    batch, q, cache = _setup(n, kv, 8, 2, 128, 16, "e4m3", seed=72)
    want, want_l, status, ws = _call(batch, q, cache)
    assert status == 0
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    try:
        mx.mx_debug_set_wait_limit_ns(0)
        mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=1, lse=lse)
        assert mx.moe_get_status(ws) in (0, mx.MX_ERR_TIMEOUT)   # a wait may be over before it is asked for
    finally:
        mx.mx_debug_set_wait_limit_ns(2_000_000_000)
    mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=1, lse=lse)
    assert mx.moe_get_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_bad_page_of_a_chunk_is_left_out(fmt, page):
    """Rows of a chunk see the other pages' keys only."""
    kv = 4 * page
    batch, q, cache = _setup([40], [kv], 8, 2, 128, page, fmt, seed=81)
    table, lens, starts = (t.clone() for t in batch.device())
    table[0, 1] = batch.pages + 5
    out, lse, status, _ = _call(batch, q, cache, dev=(table, lens, starts), causal=False)
    assert status == mx.MX_ERR_DEVICE_ARG
    less = ref.Batch([40], [kv - page], page, batch.pages, torch.cat([batch.table[:, :1], batch.table[:, 2:4]], 1))
    tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    o, l, tol, tol_l = ref.attention(q.cpu(), *tables, fmt, less, 128 ** -0.5, False, 0)
    assert torch.all((out.cpu().double() - o).abs() <= tol) and torch.all((lse.cpu().double() - l).abs() <= tol_l)


@pytest.mark.parametrize("rows", [15, 16, 17, 33, 48, 64, 65, 127, 129, 255, 257])
def test_row_counts_at_the_tiles_edges(rows):
    """One query head of its own KV head: new tokens are rows."""
    _check([rows, 1], [rows + 70, 100], 2, 2, 64, 16, seed=90 + rows)


@pytest.mark.parametrize("n,kv", [([1, 2], [90, 300]), ([70], [260]), ([40, 1, 3], [40, 200, 64])])
def test_queries_that_are_not_finite(n, kv):
    """An infinity or NaN in a query makes its own row NaN and leaves the others alone."""
    batch, q, cache = _setup(n, kv, 8, 2, 128, 16, "e4m3", seed=61)
    clean, bad = q.clone(), q.clone()
    last = batch.T - 1
    bad[0, 0, 3], bad[last, 5, 127], bad[last // 2, 6, 64] = float("inf"), float("nan"), float("-inf")
    for t, h in ((0, 0), (last, 5), (last // 2, 6)):
        clean[t, h] = 0.0
    want, want_l, status, _ = _call(batch, clean, cache)
    assert status == 0
    out, lse, status, _ = _call(batch, bad, cache)
    assert status == 0
    hit = torch.zeros(batch.T, 8, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (last, 5), (last // 2, 6)):
        hit[t, h] = True
    assert torch.all(torch.isnan(out[hit])) and torch.all(torch.isnan(lse[hit]))
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_l[~hit])


def test_many_sequences_of_all_kinds():
    """More sequences than are looked at together, of all kinds: none, single
    tokens, drafts, chunks of one and of several tiles."""
    g = torch.Generator().manual_seed(71)
    n = [[0, 1, 1, 1, 4, 1, 9, 40][int(i)] for i in torch.randint(0, 8, (300,), generator=g)]
    n[7], n[131], n[299] = 90, 200, 70
    kv = [a + int(b) for a, b in zip(n, torch.randint(0, 60, (300,), generator=g))]
    _check(n, kv, 8, 2, 64, 16, seed=72)


@pytest.mark.parametrize("rows", [24, 32, 120, 128, 136, 256])
def test_row_counts_at_the_rule_between_the_kernels(rows):
    _check([rows // 8], [rows // 8 + 130], 8, 1, 64, 16, seed=81)              # few pairs
    _check([rows // 8, 1] * 9, [rows // 8 + 30, 70] * 9, 8, 1, 64, 16, seed=82)  # many


@pytest.mark.parametrize("n,kv", [([400] * 6, [400] * 6), ([330, 90, 200], [900, 90, 1400]), ([40], [3000])])
def test_segments_that_are_split_or_not(n, kv):
    """Prompts whose tiles are about as long as a CTA's stretch."""
    _check(n, kv, 4, 2, 64, 16, seed=91)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dim", [64, 128])
def test_waits_of_chunks_that_run_out(fmt, dim):
    """A limit of zero makes waits run out for some lanes of a warp and not for
    others, again and again: each call ends, reports it, and leaves a workspace
    with which the next one is right."""
    n, kv = [90, 300], [2700, 333]
    batch, q, cache = _setup(n, kv, 8, 2, dim, 16, fmt, seed=73)
    want, want_l, status, ws = _call(batch, q, cache)
    assert status == 0
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    for _ in range(5):
        try:
            mx.mx_debug_set_wait_limit_ns(0)
            mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
            assert mx.moe_get_status(ws) == mx.MX_ERR_TIMEOUT
        finally:
            mx.mx_debug_set_wait_limit_ns(2_000_000_000)
        mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
        assert mx.moe_get_status(ws) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("n,kv", [([1] * 9, [900] * 9), ([1] * 24, [9000] * 24), ([3] * 70, [150] * 70)])
def test_waits_of_few_rows_that_run_out(n, kv, fmt):
    """The same of the few-rows kernel, with fewer units a CTA than it fetches ahead,
    with many, and with many short segments."""
    batch, q, cache = _setup(n, kv, 8, 2, 128, 16, fmt, seed=74)
    want, want_l, status, ws = _call(batch, q, cache)
    assert status == 0
    out, lse = torch.empty_like(want), torch.empty_like(want_l)
    for _ in range(5):
        try:
            mx.mx_debug_set_wait_limit_ns(0)
            mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
            assert mx.moe_get_status(ws) == mx.MX_ERR_TIMEOUT
        finally:
            mx.mx_debug_set_wait_limit_ns(2_000_000_000)
        mx.mx_paged_attention(q, cache, *batch.device(), out, ws, max_q_len=max(n), lse=lse)
        assert mx.moe_get_status(ws) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("window", [1, 3, 2 ** 31 - 1])
@pytest.mark.parametrize("n,kv", [([5, 1, 3], [2, 0, 3]), ([90, 70, 40], [30, 0, 100])])
def test_windows_over_more_new_tokens_than_keys(n, kv, window):
    """The first new tokens lie at negative positions, the window is up to an int's largest."""
    for dim in (64, 128):
        _check(n, kv, 4, 2, dim, 16, window=window, seed=101)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("n,kv,dim", [([1, 2], [90, 300], 128), ([3], [70], 64), ([70], [260], 128), ([90, 80], [90, 200], 64)])
def test_scales_that_are_nan(n, kv, dim, fmt, which):
    """A scale byte of 255 in one block of one key or value: the rows that see it are
    NaN in both kernels, those of other heads and sequences keep their bits, and, for
    a key's, those that do not see it."""
    batch, q, cache = _setup(n, kv, 8, 2, dim, 16, fmt, seed=111)
    want, want_l, status, _ = _call(batch, q, cache)
    assert status == 0
    pos = kv[0] - (n[0] + 1) // 2          # some new tokens of sequence 0 see it, in a chunk some do not
    (page,), (at,) = batch.places(0, torch.tensor([pos]))
    scales = {"k": cache.k_scales, "v": cache.v_scales}[which]
    scales[page, 1, at, dim // 32 - 1] = 255
    out, lse, status, _ = _call(batch, q, cache)
    assert status == 0
    seen = torch.zeros(batch.T, 8, dtype=torch.bool, device="cuda")
    seen[n[0] - (kv[0] - pos): n[0], 4:] = True
    assert torch.all(torch.isnan(out[seen])) and torch.all(torch.isnan(lse[seen]))
    same = ~seen
    if which == "v":
        same[: n[0], 4:] = False           # what a masked value holds may reach them
    assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_l[same])


def _bounded(q, tables, fmt, batch, scale):
    """(out, lse, their bounds), fp64, causal, with what the header states of the
    second product's roundings, element by element:
    out goes to bf16 (2^-8); a weight to f16 (2^-11), or to bf16 (2^-8) where the V scales of a
    64-key unit spread over more than 2^15; a weight times its value's largest block
    scale is held to 2^-25 of the row's largest such product (f16's smallest step,
    halved).  For few rows a key's or value's element is held to 2^-25 of its token's
    largest block scale and is zero where its own block's scale lies 2^25 below (E2M1:
    2^31).  A score sums D products in fp32 (2^-24 each of the sum of their sizes); a
    query's element is held to 2^-22 of its block's largest.  Exponents are taken in
    fp32: 2^-22 of the scores' sizes, and 2^-20 for the rest.  Only the scores' errors
    against the largest weight's count; a weight that is off by r moves out by r (v - o)
    and at most twice that once all are normalised, while they add up to less than 1/2."""
    two = torch.tensor(2.0, dtype=torch.float64)
    gone = 25 if fmt == "e4m3" else 31

    def held(x, scales):
        """How far each element of x [kv, Hk, D] may be off for its token's other blocks."""
        top = scales.double().amax(-1, keepdim=True)
        far = (scales.double() <= top - gone).repeat_interleave(32, -1)
        return torch.where(far, x.abs(), torch.minimum(x.abs(), 2.0 ** -25 * torch.pow(two, top - 127)))

    T, Hq, D = q.shape
    Hk = tables[0].shape[1]
    out, tol = (torch.zeros(T, Hq, D, dtype=torch.float64) for _ in range(2))
    lse, tol_lse = (torch.zeros(T, Hq, dtype=torch.float64) for _ in range(2))
    for b, (n, kv) in enumerate(zip(batch.n, batch.kv)):
        page, at = batch.places(b, torch.arange(kv))
        kc, ks, vc, vs = (t[page, :, at] for t in tables)
        K, V = ref.decode(kc, ks, fmt), ref.decode(vc, vs, fmt)
        v_top = vs.double().amax(-1) - 127          # [kv, Hk]
        K_off, V_off = held(K, ks), held(V, vs)
        for i in range(n):
            hi = kv - n + i + 1
            unit = torch.arange(hi) // 64
            for h in range(Hq):
                g = h * Hk // Hq
                k, v, e = K[:hi, g], V[:hi, g], v_top[:hi, g]
                x = q[batch.starts[b] + i, h].double()
                block = x.abs().unflatten(0, (-1, 32)).amax(1).repeat_interleave(32)
                s = k @ x * scale
                ds = scale * (D * 2.0 ** -24 * (k.abs() @ x.abs()) + K_off[:hi, g] @ x.abs() + 2.0 ** -22 * (k.abs() @ block))
                ds = ds + 2.0 ** -22 * (s.abs() + s.abs().max()) + 2.0 ** -20
                p, star = torch.softmax(s, 0), int(s.argmax())
                o = p @ v
                r = torch.exp(torch.log_softmax(s, 0) + ds + ds[star]) - p   # of each weight
                r[star] = 0
                assert float(r.sum()) < 0.5
                tops = torch.stack([v_top[u * 64: (u + 1) * 64, g].max() for u in range(int(unit[-1]) + 1)])
                lows = torch.stack([vs[u * 64: (u + 1) * 64, g].double().min() - 127 for u in range(int(unit[-1]) + 1)])
                half = torch.where(tops - lows > 15, 2.0 ** -8, 2.0 ** -11)[unit]
                most = (p * torch.pow(two, tops[unit])).max()
                err = (2 * r @ (v - o).abs() + (p * half) @ v.abs() + p @ V_off[:hi, g]
                       + 2.0 ** -25 * most * (torch.pow(two, -e) @ v.abs()))
                t = batch.starts[b] + i
                out[t, h], tol[t, h] = o, 2.0 ** -8 * (o.abs() + err) + err
                lse[t, h] = torch.logsumexp(s, 0)
                tol_lse[t, h] = ds[star] + 2 * r.sum() + 2.0 ** -22 * (1 + lse[t, h].abs()) + 2.0 ** -20
    return out, lse, tol, tol_lse


@pytest.mark.parametrize("spread", [4, 8, 12, 16])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("n,kv,dim", [([2, 1], [150, 40], 128), ([3], [90], 64), ([50], [150], 128), ([70], [100], 64)])
def test_tokens_that_are_large_in_one_block(n, kv, dim, fmt, spread):
    """One token of each sequence has keys and values 2^spread larger in one block of
    32; half of the query heads have zeros there, so that their scores are ordinary."""
    heads, kv_heads, page = 4, 2, 16
    batch = ref.make_batch(n, kv, page, 121)
    full = ref.Batch(list(kv), list(kv), page, batch.pages, batch.table)
    g = torch.Generator().manual_seed(122)
    k, v = (torch.randn(full.T, kv_heads, dim, generator=g) for _ in range(2))
    for b in range(len(n)):
        at = full.starts[b] + kv[b] // 3
        k[at, :, 32:] *= 2.0 ** spread
        v[at, :, 32:] *= 2.0 ** spread
    q = torch.randn(batch.T, heads, dim, generator=g)
    q[:, ::2, 32:] = 0
    q = q.to(torch.bfloat16)
    cache = mx.KVCache(batch.pages, page, kv_heads, dim, fmt)
    ws = mx.alloc_workspace(256)
    mx.mx_kv_append(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), *full.device(), ws)
    out, lse, status, _ = _call(batch, q.cuda(), cache)
    assert status == 0
    tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    o, l, tol, tol_l = _bounded(q, tables, fmt, batch, dim ** -0.5)
    assert torch.all((out.cpu().double() - o).abs() <= tol)
    assert torch.all((lse.cpu().double() - l).abs() <= tol_l)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("n,kv,page", [([1, 2], [70001, 40003], 16), ([1], [140000], 64), ([40], [66007], 16)])
def test_long_contexts(n, kv, page, fmt):
    """Thousands of pages of one sequence."""
    _check(n, kv, 2, 1, 64, page, fmt, seed=131)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,window", [([6, 3, 10, 1], 0), ([12] * 4, 0), ([12] * 4, 70), ([4, 12, 0, 9], 0)])
def test_narrow_and_wide_block_tables(n, window, dim, fmt):
    """A wider table moves sequences of a few tiles of rows from the few-rows kernel to
    the chunk kernel; what lies beyond the lengths is not looked at."""
    kv = [a + 40 + 30 * b for b, a in enumerate(n)]
    batch, q, cache = _setup(n, kv, 32, 4, dim, 16, fmt, seed=141)
    table, lens, starts = batch.device()
    wide = torch.full((len(n), 12000), -5, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    for t in (table, wide):
        out, lse, status, _ = _call(batch, q, cache, dev=(t, lens, starts), window=window)
        assert status == 0
        _compare(batch, q, cache, out, lse, fmt, dim ** -0.5, True, window)


@pytest.mark.parametrize("max_q_len,causal", [(4096, False), (1, True)])
def test_starts_that_give_the_same_tokens_to_many_sequences(max_q_len, causal):
    """Starts that fall and rise again may ask for more work than the kernels' 32-bit
    line holds: 50000 sequences of 4096 new tokens here, or, with one new token, none.
    The call is reported and writes nothing."""
    n, T, page = 100001, 4096, 65536
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = T
    cache = mx.KVCache(1, page, 1, 64)
    q = torch.randn(T, 16, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    lse = torch.full((T, 16), 3.0, device="cuda")
    ws = mx.alloc_workspace(mx.mx_paged_attention_workspace_size(T, n, 16, 1, 64, max(max_q_len, 2)))
    table = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), page, dtype=torch.int32, device="cuda")
    mx.mx_paged_attention(q, cache, table, lens, starts, out, ws, causal=causal, max_q_len=max_q_len, lse=lse)
    assert mx.moe_get_status(ws) == mx.MX_ERR_DEVICE_ARG
    assert torch.all(out == 3.0) and torch.all(lse == 3.0)
    # and the workspace is ready for a call that is right
    lens[0], starts[1:] = 300, 2
    mx.mx_paged_attention(q, cache, table, lens, starts, out, ws, causal=causal, max_q_len=max(max_q_len, 2), lse=lse)
    assert mx.moe_get_status(ws) == 0
    assert torch.all(out[:2] == 0) and torch.all(out[2:] == 3.0) and torch.all(lse[:2] != 3.0)   # a cache of zeros
