"""The decoder block's host side: its workspaces and their status words (no GPU needed)."""
import pytest
import torch

from block_scaled_mx_gb300 import block as B
from block_scaled_mx_gb300 import mxmoe as mx


@pytest.fixture
def blk(monkeypatch):
    """A block whose workspaces are host tensors and whose status words are read and
    cleared there."""

    def status(ws, stream=None):
        v = int(ws[0])
        ws[:4] = 0
        return v

    monkeypatch.setattr(mx, "alloc_workspace", lambda n, device="cpu": torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(mx, "moe_get_status", status)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(mx, "current_stream", lambda: 1, raising=False)
    return B.DecoderBlock(*[None] * 6, 8, 2, 64)


@pytest.mark.parametrize("name", ["attention", "router", "permute", "experts"])
def test_an_error_is_kept_when_a_workspace_grows(blk, name):
    for other in ("attention", "router", "permute", "experts"):
        blk._workspace(other, 256)
    blk._workspace(name, 256)[:8] = 6       # the status word, and a counter beside it
    grown = blk._workspace(name, 1024)
    assert grown.nbytes == 1024 and int(grown[4:].max()) == 0
    assert blk.status() == 6
    assert blk.status() == 0


def test_streams_have_workspaces_of_their_own(blk, monkeypatch):
    one = blk._workspace("attention", 256)
    monkeypatch.setattr(mx, "current_stream", lambda: 2, raising=False)
    two = blk._workspace("attention", 256)
    assert two is not one and blk._workspace("attention", 256) is two
    monkeypatch.setattr(mx, "current_stream", lambda: 1, raising=False)
    assert blk._workspace("attention", 256) is one
    one[:4] = 3                             # an error on either stream is found
    assert blk.status() == 3


def test_captured_graphs_have_workspaces_of_their_own(blk, monkeypatch):
    """Captures on one stream, as torch's default capture stream, one after the other: what a
    graph uses is neither another graph's nor an eager call's, and is never given up."""
    monkeypatch.setattr(mx, "alloc_captured_workspace", lambda n: torch.zeros(n, dtype=torch.uint8), raising=False)
    capture = 0
    monkeypatch.setattr(mx, "current_capture", lambda: capture, raising=False)
    eager = blk._workspace("attention", 256)
    capture = 5
    one = blk._workspace("attention", 256)
    assert blk._workspace("attention", 200) is one
    grown = blk._workspace("attention", 1024)
    capture = 8
    two = blk._workspace("attention", 256)
    capture = 0
    assert blk._workspace("attention", 256) is eager
    larger = blk._workspace("attention", 512)
    assert len({ws.data_ptr() for ws in (eager, one, grown, two, larger)}) == 5
    for ws in (one, grown, two, larger):    # an error in any of them is found
        ws[:4] = 3
        assert blk.status() == 3 and blk.status() == 0
