"""One workspace for calls of different sizes: a serving loop allocates for its
largest step and goes through steps of other sizes with it.  What one call
leaves there must not reach the next."""
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
