"""The operators together: a decoder block over a ragged batch, a step of prompts
and then steps of single tokens beside a chunk, each stage against its reference
given what the stage before it left."""
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


@pytest.mark.parametrize("fmt,cache_fmt,window", [("e4m3", "e4m3", 0), ("e2m1", "e2m1", 24)])
def test_block_over_a_ragged_batch(fmt, cache_fmt, window):
    H, I, E, k, hq, hk, d, page = 256, 128, 8, 2, 8, 2, 64, 16
    blk = B.random_block(H, I, E, k, hq, hk, d, fmt=fmt, window=window, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    kv = [0, 0, 0]
    full = ref.make_batch([1, 1, 1], [90, 40, 20], page, 5)
    cache = mx.KVCache(full.pages, page, hk, d, cache_fmt)
    for new in ([70, 1, 9], [1, 1, 1], [12, 1, 0]):
        kv = [a + b for a, b in zip(kv, new)]
        batch = ref.Batch(new, list(kv), page, full.pages, full.table)
        x = torch.randn(batch.T, H, generator=g, device="cuda")
        res = torch.randn(batch.T, H, generator=g, device="cuda").to(torch.bfloat16)
        out, after = blk.forward(x, res, cache, *batch.device(), max(new))
        assert blk.status() == 0
        s = blk.last
        # attention, from the queries and what the cache holds
        tables = [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        o, _, tol, _ = ref.attention(s["q"].cpu(), *tables, cache_fmt, batch, d ** -0.5, True, window)
        assert torch.all((s["att"].cpu().double() - o).abs() <= tol)
        # the residual stream: two fp32 additions, each rounded to bf16
        mid = (x.cpu() + res.cpu().float()).to(torch.bfloat16)
        proj = s["att"].view(batch.T, hq * d) @ blk.w_o.t()
        want = (proj.cpu().float() + mid.float()).to(torch.bfloat16)
        assert torch.equal(after.cpu(), want)
        # the norm's codes hold y: to half a step of e4m3 (2^-4) or of the block's smallest
        y, codes = s["y"].cpu().double(), ref.decode(s["codes"].cpu(), s["scales"].cpu(), "e4m3")
        low = torch.exp2(s["scales"].cpu().double() - 127 - 10).repeat_interleave(32, 1)
        # y is rounded to bf16 (2^-8) beside; a block's largest may saturate at 448 / 512
        assert torch.all((codes - y).abs() <= (2.0 ** -4 + 2.0 ** -8) * y.abs() + low + (y.abs() - codes.abs()).clamp(min=0)
                         * (codes.abs() >= 448 * torch.exp2(s["scales"].cpu().double() - 127).repeat_interleave(32, 1)))
        # the experts: the layer in one call on the same activations (a code times its
        # scale has four significant bits and is quantised to itself).  An h next to a
        # rounding border may take either code, a step of at most 2^-3: one in 1000
        # of them moves the output by 2^-3 / 1000^0.5 = 0.004 (relative, L2)
        logits = torch.empty(batch.T, E, dtype=torch.float32, device="cuda")
        mx.moe_route_gemm_topk(s["y"], blk.w_router, k, mx.alloc_workspace(256 + 4 * 128 * E), logits=logits)
        one = blk.experts.forward(codes.to(torch.bfloat16).cuda(), logits)
        assert float((out - one).norm() / one.norm()) <= 0.004


def test_example_runs(capsys):
    B.main(prompts=(40, 3), steps=2, H=256, I=128, E=4, k=2, n_heads=4, n_kv_heads=1, head_dim=64, page=16)
    assert "step 2" in capsys.readouterr().out


def test_block_keeps_nothing_of_a_call():
    """Unless it is asked to: a call's activations are free once it has returned."""
    args = (256, 128, 8, 2, 8, 2, 64)
    blk = B.random_block(*args, keep_last=False)
    batch = ref.make_batch([2000], [2000], 16, 1)
    x = torch.randn(2000, 256, device="cuda")
    res = torch.zeros(2000, 256, dtype=torch.bfloat16, device="cuda")
    cache = mx.KVCache(batch.pages, 16, 2, 64)
    dev = batch.device()
    out, after = blk.forward(x, res, cache, *dev, 2000)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out, after = blk.forward(x, res, cache, *dev, 2000)
    torch.cuda.synchronize()
    # less than one of the kept tensors more (a reused block may be larger than asked for)
    assert blk.last is None and torch.cuda.memory_allocated() - before < 2000 * 12 * 64 * 2
    w = blk.__dict__
    plain = B.DecoderBlock(*(w[n] for n in ("w_qkv", "w_o", "g_attn", "g_mlp", "w_router", "experts", "n_heads", "n_kv_heads",
                                            "head_dim")))
    plain.forward(x, res, cache, *dev, 2000)
    assert plain.last is None


def test_calls_of_one_block_on_two_streams():
    """Steps of different batches that overlap give what they give one after the other."""
    blk = B.random_block(256, 128, 8, 2, 8, 2, 64, keep_last=False)
    g = torch.Generator(device="cuda").manual_seed(9)
    steps = []
    for new in ([700, 60], [1] * 40):
        batch = ref.make_batch(new, [n + 300 for n in new], 16, 1)
        cache = mx.KVCache(batch.pages, 16, 2, 64)
        steps.append((torch.randn(batch.T, 256, generator=g, device="cuda"),
                      torch.randn(batch.T, 256, generator=g, device="cuda").to(torch.bfloat16), cache, *batch.device(), max(new)))
    want = [[blk.forward(*s) for s in steps] for _ in range(2)][1]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(blk.forward(*steps[i]))
    assert blk.status() == 0
    for i in range(2):
        for out, after in got[i]:
            assert torch.equal(after, want[i][1])
            # a token's k + 1 = 3 slots in pieces, added in any order: at most 16
            # additions of 2^-24 each, of terms that sum to four times their sum's size
            assert float((out - want[i][0]).norm()) <= 2.0 ** -18 * float(want[i][0].norm())


def test_block_without_tokens():
    """A step in which no sequence has a new token."""
    blk = B.random_block(256, 128, 8, 2, 8, 2, 64, keep_last=False)
    batch = ref.Batch([0, 0], [7, 0], 16, 4, torch.tensor([[0], [1]], dtype=torch.int32))
    x = torch.empty(0, 256, device="cuda")
    out, after = blk.forward(x, x.to(torch.bfloat16), mx.KVCache(4, 16, 2, 64), *batch.device(), 0)
    assert out.shape == after.shape == (0, 256) and blk.status() == 0
