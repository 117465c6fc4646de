"""One workspace for calls of different sizes: a serving loop allocates for its
largest step and goes through steps of other sizes with it.  What one call
leaves there must not reach the next."""
import ctypes

import numpy as np
import pytest
import torch

from block_scaled_mx_gb300 import block as B
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


def _permuted(ids, E):
    """counts, offsets and slots of ids [T, k] from the definition."""
    T, k = ids.shape
    with_shared = np.concatenate([ids, np.full((T, 1), E)], 1).reshape(-1)
    counts = np.bincount(with_shared, minlength=E + 1)
    return counts, np.concatenate([[0], np.cumsum(counts)]), np.argsort(with_shared, kind="stable")


@pytest.mark.parametrize("E,k", [(16, 4), (128, 8)])
def test_permute_of_other_sizes_on_one_workspace(E, k):
    rng = np.random.default_rng(E)
    sizes = [2000, 1500, 700, 400, 257, 256, 6, 1, 300, 1999, 2000]
    ws = mx.alloc_workspace(mx.moe_permute_workspace_size(max(sizes), E, k))
    for T in sizes:
        ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
        counts, offsets, order = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E + 1, E + 2, T * (k + 1)))
        mx.moe_permute(torch.from_numpy(ids).cuda(), E, counts, offsets, order, ws)
        assert mx.moe_get_status(ws) == 0
        for got, want in zip((counts, offsets, order), _permuted(ids, E)):
            assert np.array_equal(got.cpu().numpy(), want), T


@pytest.mark.parametrize("separate", ["0", "1"])
def test_layer_of_other_sizes_on_one_workspace(separate, monkeypatch):
    """moe_forward through one layer object, whose workspace grows and stays.  Two
    calls differ in the order in which a token's k + 1 = 5 slots, each in a few pieces,
    are added in fp32: at most 16 additions of 2^-24 each, of terms whose sizes sum
    to four times their sum's at most."""
    monkeypatch.setenv("MXMOE_SEPARATE_PERMUTE", separate)
    H, I, E, k = 256, 128, 32, 4
    layer = B.random_block(H, I, E, k, 4, 2, 64, seed=1).experts
    g = torch.Generator(device="cuda").manual_seed(2)
    for T in (1500, 6, 128, 40, 256, 6, 700, 300, 128, 1, 1500):
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        logits = torch.randn(T, E, generator=g, device="cuda")
        out = layer.forward(x, logits)
        assert mx.moe_get_status(layer.workspace(T)) == 0
        fresh = torch.empty_like(out)
        ws = mx.alloc_workspace(mx.moe_workspace_size(T, H, I, E, k, layer.fmt))
        mx.moe_forward(x, logits, layer.w1, layer.w2, layer.fmt, I, k, fresh, ws)
        assert float((out - fresh).norm()) <= 2.0 ** -18 * float(fresh.norm()), T


def test_block_of_other_sizes():
    """The decoder block's steps: prompts, then shorter ones, then single tokens."""
    H, I, E, k, hq, hk, d, page = 256, 128, 8, 2, 8, 2, 64, 16
    blk = B.random_block(H, I, E, k, hq, hk, d, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    full = ref.make_batch([1, 1], [900, 900], page, 5)
    for new in ([600, 100], [1, 1], [300, 100], [1, 0], [257, 1], [500, 250]):
        batch = ref.Batch(new, list(new), page, full.pages, full.table)
        x = torch.randn(batch.T, H, generator=g, device="cuda")
        res = torch.randn(batch.T, H, generator=g, device="cuda").to(torch.bfloat16)
        out, after = blk.forward(x, res, mx.KVCache(full.pages, page, hk, d), *batch.device(), max(new))
        assert blk.status() == 0
        again = B.random_block(H, I, E, k, hq, hk, d, seed=3)   # the same weights, its own workspaces
        want, want_after = again.forward(x, res, mx.KVCache(full.pages, page, hk, d), *batch.device(), max(new))
        assert torch.equal(after, want_after)
        assert float((out - want).norm()) <= 2.0 ** -18 * float(want.norm()), new


def _step(blk, new, lens, seed, hk=2, d=64, page=16):
    """A step of a block on tensors of its own: (run it, its outputs' (out, after) by a block
    of the same weights that nothing was captured from)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = ref.make_batch([1] * len(new), [900] * len(new), page, seed)
    batch = ref.Batch(new, lens, page, full.pages, full.table)
    x = torch.randn(batch.T, 256, generator=g, device="cuda")
    res = torch.randn(batch.T, 256, generator=g, device="cuda").to(torch.bfloat16)
    past = torch.randint(0, 120, (2, full.pages, hk, page, d), generator=g, device="cuda", dtype=torch.uint8)
    metadata = batch.device()

    def run(block):
        cache = mx.KVCache(full.pages, page, hk, d)
        cache.k_codes.copy_(past[0]), cache.v_codes.copy_(past[1])
        cache.k_scales.fill_(122), cache.v_scales.fill_(122)
        return lambda: block.forward(x, res, cache, *metadata, max(new))

    return run(blk), run(B.random_block(256, 128, 8, 2, 8, hk, d, seed=3, projections="e2m1", rope=mx.Rope(d)))()


def _same(got, want):
    # the experts' slots are added in any order: see test_layer_of_other_sizes_on_one_workspace
    return torch.equal(got[1], want[1]) and float((got[0] - want[0]).norm()) <= 2.0 ** -18 * float(want[0].norm())


def test_graphs_of_one_block_run_in_any_order_and_side_by_side():
    """Two graphs captured one after the other on torch's capture stream, of calls of different
    sizes: either runs alone, first or beside the other."""
    blk = B.random_block(256, 128, 8, 2, 8, 2, 64, seed=3, projections="e2m1", rope=mx.Rope(64))
    steps = [_step(blk, [1] * 5, [700, 3, 64, 900, 129], 7), _step(blk, [30, 1, 400], [600, 800, 400], 8)]
    steps[0][0]()   # what a first call sets up once
    graphs, outs = [torch.cuda.CUDAGraph() for _ in steps], []
    for graph, (run, _) in zip(graphs, steps):
        with torch.cuda.graph(graph):
            outs.append(run())
    assert blk.status() == 0            # of graphs that have not run yet
    streams = [torch.cuda.Stream() for _ in graphs]
    for order in ([1], [0], [0, 1] * 20):
        for out, after in outs:
            out.fill_(float("nan")), after.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in order:
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert blk.status() == 0 and all(_same(outs[i], steps[i][1]) for i in order)


def test_a_graph_outlives_the_workspaces_of_its_stream():
    """A graph captured on a stream that eager calls use too, the workspaces of which grow."""
    blk = B.random_block(256, 128, 8, 2, 8, 2, 64, seed=3, projections="e2m1", rope=mx.Rope(64))
    (small, want), (large, want_large) = _step(blk, [1] * 4, [700, 3, 64, 900], 7), _step(blk, [300, 1, 400], [600, 800, 400], 8)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        small()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = small()
        grown = large()                 # a larger call of the same capture
        again = small()
    with torch.cuda.stream(stream):
        assert _same(large(), want_large)
        filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (256, 4096, 70000, 1 << 20, 5 << 20, 41 << 20)]
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert blk.status() == 0 and _same(out, want) and _same(again, want) and _same(grown, want_large)
    assert all(int(f.min()) == 255 for f in filled)
    assert mx.capture_id() == 0 and mx.current_capture() == 0


def test_a_workspace_is_zero_before_its_graph_runs():
    x, graph = torch.ones(64, device="cuda"), torch.cuda.CUDAGraph()
    ids = set()
    with torch.cuda.graph(graph):
        ids.add(mx.current_capture())
        y = x + 1
        workspaces = [mx.alloc_captured_workspace(n) for n in (5000, 1, 50 << 20)]
        z = y + 1
    for ws in workspaces:
        assert int(ws.max()) == 0
        ws.fill_(7)
    graph.replay()
    assert all(int(ws.min()) == 7 for ws in workspaces) and torch.all(z == 3)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        ids.add(mx.current_capture())
        x + 1
    assert len(ids) == 2 and 0 not in ids
    mode = ctypes.c_int(0)
    assert mx.lib().mx_exchange_capture_mode(ctypes.addressof(mode)) == 0 and mode.value == 0   # as it was
