"""Chunk attention and the windowed decode without a GPU: refusals and workspace sizes."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_binding_checks import Dev
from tests.test_serving_abi import INVALID, UNSUPPORTED, dev, heads, heads_struct, kvq  # noqa: F401  (a fixture)

TOO_SMALL = 3


def views_of(kvq, n=1, d=128, hkv=2, fmt=("fp16", "fp16", 0, 0), pages=8, table=None, **kw):
    arr = (kvq.KvqTierView * n)()
    keep = []
    for v in arr:
        signs = np.ones((hkv, d), dtype=np.int8)
        cache = kvq.PagedCache(d, hkv, pages, fmt[0], fmt[1], fmt[2], fmt[3], signs, signs, device="cpu")
        s = cache.struct
        # addresses that are never read
        s.k_rows, s.v_rows, s.k_signs, s.v_signs = (1 << 12,) * 4
        if s.k_aux:
            s.k_aux = s.v_aux = 1 << 12
        for name, x in kw.items():
            setattr(s, name, x)
        keep.append(cache)
        v.cache = ctypes.pointer(s)
        v.block_table, v.seq_lens, v.max_pages = 1 << 12, 1 << 12, pages if table is None else table
    return arr, keep


def chunk(kvq, arr, n, q=None, offsets=1 << 12, batch=3, tokens=10, window=0, sinks=0, ws=1 << 12, size=1 << 40,
          status=None, visible=True):
    q = heads_struct(kvq, x=1 << 12, out=1 << 13, n=4, xt=512, ot=512) if q is None else q
    v = kvq.KvqVisible(window, sinks)
    return kvq.lib().kvq_chunk_attention(arr, n, bytes(q) if q else None, offsets, batch, tokens,
                                         ctypes.byref(v) if visible else None, ws, size, status, None)


def test_chunk_refusals(kvq):
    arr, keep = views_of(kvq)
    n = kvq.kvq_kernel_launches()
    assert chunk(kvq, arr, 1, batch=0) == 0 and chunk(kvq, arr, 1, tokens=0) == 0  # nothing to do
    assert chunk(kvq, arr, 1, batch=0, tokens=0, ws=None, size=0) == 0
    assert chunk(kvq, arr, 1, size=0) == TOO_SMALL and chunk(kvq, arr, 1, size=0, visible=False) == TOO_SMALL
    for bad in (dict(batch=-1), dict(tokens=-1), dict(window=-1), dict(sinks=-1, window=4), dict(sinks=2), dict(ws=None),
                dict(ws=(1 << 12) + 128), dict(offsets=(1 << 12) + 2), dict(status=(1 << 12) + 2),
                dict(offsets=None, batch=3, tokens=10)):
        assert chunk(kvq, arr, 1, **bad) == INVALID, bad
    for bad in (dict(x=0), dict(out=0), dict(x=(1 << 12) + 8), dict(out=(1 << 13) + 2), dict(n=0), dict(xt=516), dict(xh=4),
                dict(ot=100), dict(oh=64), dict(xt=-8), dict(n=3), dict(n=5)):
        h = heads_struct(kvq, **{**dict(x=1 << 12, out=1 << 13, n=4, xt=512, ot=512), **bad})
        assert chunk(kvq, arr, 1, q=h) == INVALID, bad
    h = heads_struct(kvq, x=1 << 12, out=1 << 13, n=6, xt=768, ot=768)
    assert chunk(kvq, arr, 1, q=h) == UNSUPPORTED  # three query heads a kv head
    assert kvq.lib().kvq_chunk_attention(arr, 1, None, 1 << 12, 3, 10, None, 1 << 12, 1 << 40, None, None) == INVALID
    assert chunk(kvq, arr, 0) == INVALID and chunk(kvq, None, 1) == INVALID
    assert chunk(kvq, arr, 1, tokens=1 << 25) == UNSUPPORTED and chunk(kvq, arr, 1, batch=65537) == UNSUPPORTED
    far, keep2 = views_of(kvq, table=(1 << 27) - 16)
    assert chunk(kvq, far, 1) == UNSUPPORTED  # positions beyond 32 bits
    many, keep3 = views_of(kvq, hkv=1 << 13)
    many[0].cache[0].num_pages = 1 << 20
    h = heads_struct(kvq, x=1 << 12, out=1 << 13, n=1 << 13, xt=1 << 20, ot=1 << 20)
    assert chunk(kvq, many, 1, q=h) == UNSUPPORTED  # rows beyond 32 bits
    for bad in (dict(k_signs=(1 << 12) + 8), dict(v_signs=(1 << 12) + 1), dict(k_rows=0), dict(v_rows=(1 << 12) + 4)):
        other, keep4 = views_of(kvq, **bad)
        assert chunk(kvq, other, 1) == INVALID, bad
    two, keep5 = views_of(kvq, 2)
    two[1].cache[0].page_size = 8
    assert chunk(kvq, two, 2) == INVALID
    arr[0].seq_lens = None
    assert chunk(kvq, arr, 1) == INVALID
    assert kvq.kvq_kernel_launches() == n


def test_window_refusals(kvq):
    arr, keep = views_of(kvq)
    n = kvq.kvq_kernel_launches()

    def call(q=1 << 12, batch=3, hq=4, window=8, sinks=1, out=1 << 13, ws=1 << 12, size=1 << 40, status=None, tiers=arr):
        v = kvq.KvqVisible(window, sinks)
        return kvq.lib().kvq_decode_attention_window(tiers, 1, q, batch, hq, ctypes.byref(v), out, ws, size, status, None)

    assert call(batch=0) == 0 and call(size=0) == TOO_SMALL
    for bad in (dict(q=None), dict(out=None), dict(q=(1 << 12) + 8), dict(out=(1 << 13) + 8), dict(batch=-1), dict(hq=0),
                dict(hq=3), dict(window=-1), dict(sinks=-1), dict(window=0, sinks=1), dict(ws=None), dict(ws=(1 << 12) + 16),
                dict(status=(1 << 12) + 1), dict(tiers=None)):
        assert call(**bad) == INVALID, bad
    assert call(hq=6) == UNSUPPORTED
    assert kvq.kvq_kernel_launches() == n


def test_workspace_sizes(kvq):
    """A window bounds what a call needs; both calls refuse a null result."""
    arr, keep = views_of(kvq, pages=1 << 14, fmt=("codebook", "codebook", 4, 4), d=256)
    n = ctypes.c_size_t()

    def size(window=0, sinks=0, tokens=64, batch=4):
        v = kvq.KvqVisible(window, sinks)
        assert kvq.lib().kvq_chunk_workspace_size(arr, 1, batch, tokens, 4, ctypes.byref(v), ctypes.byref(n)) == 0
        return n.value

    assert size(window=512, sinks=4) < size() / 8
    assert size(tokens=64) <= size(tokens=65) and size(batch=4) < size(batch=5)
    assert size(tokens=0) >= 0 and size(batch=0) >= 0
    f = kvq.lib()
    assert f.kvq_chunk_workspace_size(arr, 1, 4, 64, 4, None, None) == INVALID
    assert f.kvq_decode_window_workspace_size(arr, 1, 4, 4, None, None) == INVALID
    assert f.kvq_decode_window_workspace_size(arr, 1, 4, 4, None, ctypes.byref(n)) == 0 and n.value > 0


class Buffer(Dev):
    def element_size(self):
        return 1


class Cache:
    class struct:
        head_dim = 128


def test_binding_refusals(kvq):
    """Tensors that the library must not be given."""
    class View:
        cache = Cache
        block_table, seq_lens = dev((3, 4), torch.int32), dev((3,), torch.int32)

    q, out, off = heads(10, 4, 128), heads(10, 4, 128), dev((4,), torch.int32)
    ws = Buffer(torch.zeros(64, dtype=torch.uint8))
    f = kvq.kvq_chunk_attention
    with pytest.raises(ValueError):
        f([], off, q, out, ws)
    for bad in (dict(q=heads(10, 4, 64)), dict(out=heads(9, 4, 128)), dict(out=heads(10, 2, 128)), dict(workspace=None),
                dict(workspace=torch.zeros(64, dtype=torch.uint8)), dict(q_offsets=dev((4, 1), torch.int32)),
                dict(q_offsets=dev((0,), torch.int32)), dict(q_offsets=dev((5,), torch.int32)),  # four sequences, three rows
                dict(q=heads(10, 128, 4).t.transpose(1, 2)), dict(window=1 << 31), dict(sinks=-(1 << 32))):
        args = {**dict(q_offsets=off, q=q, out=out, workspace=ws), **bad}
        with pytest.raises((ValueError, TypeError)):
            f([View], **args)
    with pytest.raises(TypeError):
        f([View], dev((4,), torch.int64), q, out, ws)
    with pytest.raises(TypeError):
        f([View], off, heads(10, 4, 128, dtype=torch.float32), out, ws)
    with pytest.raises(TypeError):
        f([View], off, q, out, ws, status=dev((1,), torch.int64))
    g = kvq.kvq_decode_attention_window
    q, out = dev((3, 4, 128), torch.float16), dev((3, 4, 128), torch.float16)
    with pytest.raises(ValueError):
        g([], q, out, ws, 8)
    with pytest.raises(TypeError):
        g([View], q, dev((3, 4, 128), torch.float32), ws, 8)
    for bad in (dict(q=dev((3, 4, 64), torch.float16)), dict(out=dev((3, 2, 128), torch.float16)),
                dict(q=dev((4, 4, 128), torch.float16), out=dev((4, 4, 128), torch.float16)), dict(workspace=None),
                dict(window=1 << 40)):
        args = {**dict(q=q, out=out, workspace=ws, window=8), **bad}
        with pytest.raises(ValueError):
            g([View], **args)
