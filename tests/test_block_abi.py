"""Host-side argument checks of the operators around the expert layer: every
call below is refused before any device work (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from block_scaled_mx_gb300 import build as B
    from block_scaled_mx_gb300 import mxmoe as mx

    B.build()
    return mx.lib()


P = ctypes.c_void_p
fake = P(4096)   # never dereferenced
odd = P(4098)


def _norm(L, x=fake, xt=0, res=fake, rt=0, w=fake, wt=0, T=4, H=64, eps=1e-6, ro=fake, y=fake, fmt=0, codes=fake,
          scales=fake):
    return L.mx_add_rmsnorm(x, xt, res, rt, w, wt, T, H, eps, ro, y, fmt, codes, scales, None)


def test_norm_refusals(L):
    assert _norm(L, T=0) == 0
    for bad in (dict(x=None), dict(w=None), dict(T=-1), dict(H=0), dict(xt=2), dict(wt=-1), dict(rt=3), dict(eps=0.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(fmt=2), dict(ro=None), dict(res=None),
                dict(scales=None), dict(codes=None), dict(y=None, codes=None, scales=None)):
        assert _norm(L, **bad) == 1, bad
    for bad in (dict(H=48), dict(H=32800)):
        assert _norm(L, **bad) == 2, bad
    for bad in (dict(x=odd), dict(res=odd), dict(w=odd), dict(ro=odd), dict(y=odd), dict(codes=odd)):
        assert _norm(L, **bad) == 3, bad


def _cache(**kw):
    from block_scaled_mx_gb300 import mxmoe as mx

    f = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, num_pages=8, page_size=16, n_kv_heads=2,
             head_dim=64, fmt=0)
    f.update(kw)
    return mx.KVCacheTables(*(f[n] for n, _ in mx.KVCacheTables._fields_))


BAD_CACHE = [(dict(num_pages=0), 1), (dict(page_size=-16), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1),
             (dict(fmt=2), 1), (dict(head_dim=80), 2), (dict(k_codes=0), 1), (dict(v_scales=0), 1), (dict(k_codes=4104), 3),
             (dict(v_scales=4098), 3), (dict(page_size=2 ** 30), 2)]


def test_cache_refusals(L):
    def append(c=None, k=fake, ks=128, v=fake, vs=128, bt=fake, kv=fake, qs=fake, n=2, mp=4, T=4, ws=fake, wb=256):
        c = _cache() if c is None else c
        return L.mx_kv_append(ctypes.addressof(c), k, ks, v, vs, bt, kv, qs, n, mp, T, ws, wb, None)

    def read(c=None, bt=fake, kv=fake, qs=fake, n=2, mp=4, T=4, ko=fake, vo=fake, ws=fake, wb=256):
        c = _cache() if c is None else c
        return L.mx_kv_read(ctypes.addressof(c), bt, kv, qs, n, mp, T, ko, vo, ws, wb, None)

    assert L.mx_kv_append(None, fake, 128, fake, 128, fake, fake, fake, 2, 4, 4, fake, 256, None) == 1
    assert L.mx_kv_read(None, fake, fake, fake, 2, 4, 4, fake, fake, fake, 256, None) == 1
    assert append(T=0) == 0 and append(n=0) == 0 and read(T=0) == 0
    for kw, want in BAD_CACHE:
        assert append(_cache(**kw), ks=4096, vs=4096) == want, kw
        assert read(_cache(**kw)) == want, kw
    for f in (append, read):
        for bad in (dict(bt=None), dict(kv=None), dict(qs=None), dict(ws=None), dict(T=-1), dict(n=-1), dict(mp=0)):
            assert f(**bad) == 1, bad
        assert f(ws=P(4112)) == 3 and f(bt=odd) == 3 and f(wb=255) == 4
    assert append(k=None) == 1 and append(v=None) == 1 and append(ks=127) == 1 and append(vs=64) == 1
    assert append(k=odd) == 3 and append(ks=132) == 3
    assert read(ko=None) == 1 and read(vo=odd) == 3


def test_attention_refusals(L):
    size = L.mx_paged_attention_workspace_size(4, 2, 8, 2, 64, 4)
    assert size > 256

    def attend(c=None, q=fake, qs=512, h=8, bt=fake, kv=fake, st=fake, n=2, mp=4, T=4, mq=4, scale=0.1, causal=1, win=0,
               out=fake, lse=fake, ws=fake, wb=size):
        c = _cache() if c is None else c
        return L.mx_paged_attention(ctypes.addressof(c), q, qs, h, bt, kv, st, n, mp, T, mq, scale, causal, win, out,
                                    lse, ws, wb, None)

    assert attend(T=0) == 0 and attend(n=0) == 0 and attend(mq=0) == 0
    for kw, want in BAD_CACHE:
        assert attend(_cache(**kw), qs=4096) == want, kw
    for bad in (dict(q=None), dict(out=None), dict(bt=None), dict(kv=None), dict(st=None), dict(ws=None), dict(h=0),
                dict(h=7), dict(qs=511), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(scale=-1.0), dict(win=-1), dict(win=4, causal=0), dict(mq=-1), dict(T=-2)):
        assert attend(**bad) == 1, bad
    assert attend(_cache(head_dim=96), qs=4096) == 2 and attend(_cache(page_size=24)) == 2
    assert attend(T=2 ** 28) == 2
    for bad in (dict(q=odd), dict(qs=516), dict(out=odd), dict(lse=odd), dict(ws=P(4352 + 16))):
        assert attend(**bad) == 3, bad
    assert attend(wb=size - 1) == 4 and attend(wb=100) == 4


def test_workspace_size_is_host_only(L):
    f = L.mx_paged_attention_workspace_size
    assert f(4, 2, 8, 3, 64, 4) == 0 and f(4, 2, 8, 2, 96, 4) == 0 and f(-1, 2, 8, 2, 64, 4) == 0
    assert f(4096, 2, 32, 8, 128, 4096) >= f(1, 1, 32, 8, 128, 1)


def test_binding_checks_tensors(L):
    from block_scaled_mx_gb300 import mxmoe as mx

    meta = dict(device="meta")
    x = torch.empty(4, 64, dtype=torch.float16, **meta)
    with pytest.raises(ValueError, match="weight"):
        mx.mx_add_rmsnorm(x, torch.empty(32, **meta), 1e-6)
    with pytest.raises(ValueError, match="codes"):
        mx._dense(torch.empty(4, 64, dtype=torch.uint8, **meta), torch.uint8, (4, 32), "codes")
    with pytest.raises(ValueError, match="residual_out"):
        mx._dense(x, torch.bfloat16, (4, 64), "residual_out")
    with pytest.raises(ValueError, match="CUDA"):
        mx.KVCache(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="k_scales"):
        t = torch.empty(4, 2, 16, 64, dtype=torch.uint8)
        mx.KVCache.of(t, t, t, t, 64)
    with pytest.raises(ValueError, match="int32"):
        mx._batch(torch.zeros(2, 3), torch.zeros(2), torch.zeros(3))
    with pytest.raises(ValueError, match="kv_lens"):
        mx._dense(torch.zeros(2, dtype=torch.int64), torch.int32, (2,), "kv_lens")
    with pytest.raises(ValueError, match="q_starts"):
        mx._dense(torch.zeros(2, dtype=torch.int32), torch.int32, (3,), "q_starts")
    with pytest.raises(ValueError, match="dense"):
        mx._rows(torch.empty(4, 64, 8, dtype=torch.bfloat16, **meta).transpose(1, 2), 8, 64, "q")
    with pytest.raises(ValueError, match="bf16"):
        mx._rows(torch.empty(4, 8, 64, **meta), 8, 64, "q")


def test_attention_refuses_work_that_its_counters_cannot_hold(L):
    """The kernels count places of work in 32 bits, and those of one KV head in a
    signed int: one head of 2^20 new tokens and 32 query heads over 2^20 keys has
    131072 tiles of 16400 places, more than 2^31 - 1.  The workspace is too small
    in every call, so that none is launched."""
    size = L.mx_paged_attention_workspace_size
    assert size(2 ** 20, 1, 32, 1, 128, 2 ** 20) > 256

    def attend(T, heads, kv_heads, keys, n=1):
        c = _cache(num_pages=keys // 64, page_size=64, n_kv_heads=kv_heads, head_dim=128)
        return L.mx_paged_attention(ctypes.addressof(c), fake, heads * 128, heads, fake, fake, fake, n, keys // 64, T, T, 0.1, 0, 0,
                                    fake, fake, fake, 256, None)

    assert attend(2 ** 20, 32, 1, 2 ** 20) == 2        # 2.15e9 places of the one head
    assert attend(2 ** 19, 64, 1, 2 ** 20) == 2
    assert attend(2 ** 20, 32, 2, 2 ** 20) == 4        # 1.07e9 of each of two
    assert attend(2 ** 19, 32, 1, 2 ** 20) == 4
    assert attend(2 ** 20, 32, 8, 2 ** 22) == 2        # 8.6e9 in all


def test_binding_imports_on_a_torch_without_cuda():
    """The binding takes the current stream's handle from names that only a CUDA
    build of torch has; without them it imports, and falls back to torch's objects."""
    import os
    import subprocess
    import sys

    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from block_scaled_mx_gb300 import mxmoe as mx\n"
            "torch.cuda.current_stream = lambda: type('S', (), {'cuda_stream': 77})()\n"
            "assert mx._stream(None) == 77 and mx._stream(5) == 5\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_binding_refuses_numbers_that_do_not_fit(L, monkeypatch):
    """ctypes drops the high bits of an int: a window of 2^32 + 5 would be one of 5."""
    from block_scaled_mx_gb300 import mxmoe as mx

    seen = []

    class Recorder:   # in the library's place, as no call may reach a device
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(mx, "_lib", Recorder())
    monkeypatch.setattr(mx, "_ptr", lambda t: 0)
    monkeypatch.setattr(mx, "_rows", lambda *a: (0, 0))
    monkeypatch.setattr(mx, "_dense", lambda *a: 0)
    cache = type("Cache", (), {"head_dim": 64, "_address": 0})()
    q, t = torch.empty(0, 8, 64), torch.empty(1, 1)

    def attend(**kw):
        mx.mx_paged_attention(q, cache, t, t, t, None, t, stream=0, **kw)

    for bad in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="window"):
            attend(window=bad)
        with pytest.raises(ValueError, match="max_q_len"):
            attend(max_q_len=bad)
        with pytest.raises(ValueError, match="max_q_len"):
            mx.mx_paged_attention_workspace_size(4, 2, 8, 2, 64, bad)
    assert not seen
    attend(window=2 ** 31 - 1, max_q_len=3)
    assert seen == ["mx_paged_attention"]


def test_attention_refuses_a_scale_that_overflows_with_log2_e(L):
    """The kernels work in powers of two: scale * log2(e) has to be finite too."""
    c = _cache()

    def attend(scale):   # with too small a workspace, so that nothing is launched
        return L.mx_paged_attention(ctypes.addressof(c), fake, 512, 8, fake, fake, fake, 2, 4, 4, 4, scale, 1, 0, fake, fake,
                                    fake, 256, None)

    assert attend(2.3e38) == 4 and attend(2.4e38) == 1 and attend(3.4e38) == 1


def test_workspace_holds_either_kernels_parts(L):
    """Which kernel takes a sequence of a few tiles of rows depends on the length that
    its block table allows, which the workspace's size does not ask for."""
    f = L.mx_paged_attention_workspace_size
    for dim in (64, 128):
        chunks = f(4096, 1, 8, 1, dim, 4096)
        for n, rows in ((16, 128), (16, 24), (1, 40), (64, 17)):
            assert f(n * rows, n, 1, 1, dim, rows) >= chunks, (n, rows)
        assert f(16 * 16, 16, 1, 1, dim, 16) < chunks
