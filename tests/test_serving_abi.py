"""The serving entry points without a GPU: the rotary table against the oracle, and argument
checks that fail before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rope as orope
from tests.test_binding_checks import Dev

KINDS = [("none", 1.0, 0.0, 0.0, 0.0), ("linear", 4.0, 0.0, 0.0, 0.0), ("base", 8.0, 0.0, 0.0, 0.0),
         ("by_parts", 8.0, 8192.0, 1.0, 32.0)]
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def kvq():
    from quantized_decode_attention_rht_gb300 import build
    build.build()
    import quantized_decode_attention_rht_gb300 as m
    m.lib()
    return m


class Heads(Dev):
    """A strided stand-in of heads."""

    def stride(self, i=None):
        return self.t.stride() if i is None else self.t.stride(i)


def dev(shape, dtype):
    return Dev(torch.zeros(shape, dtype=dtype))


def heads(*shape, dtype=torch.float16):
    return Heads(torch.zeros(shape, dtype=dtype))


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("kind,factor,context,low,high", KINDS)
def test_table_matches_oracle(kvq, rot, kind, factor, context, low, high):
    t = kvq.kvq_rope_table(10000.0, rot, kind, factor, context, low, high)
    w = orope.frequencies(10000.0, rot, kind, factor, context, low, high)
    want = np.array([int(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) for x in w], dtype=object)
    # pow and the scaling's few operations: a few units in the last of 53 bits
    for got, x in zip(t.tolist(), want):
        assert abs(int(got) - x) <= 16 * 2.0 ** -53 * x + 1


def test_table_wraps_whole_turns(kvq):
    # base below 1 gives pairs that turn more than once per token; whole turns do not matter
    t = kvq.kvq_rope_table(0.001, 4)
    w = orope.frequencies(0.001, 4)
    assert w[1] > 2 * math.pi
    assert abs(int(t[1]) / 2.0 ** 64 - math.fmod(w[1] / (2 * math.pi), 1.0)) < 1e-14


def test_table_refusals(kvq):
    for args in [(0.0, 64), (-1.0, 64), (math.inf, 64), (math.nan, 64), (1e4, 0), (1e4, 3), (1e4, 258), (1e4, -2),
                 (1e4, 64, 4), (1e4, 64, -1), (1e4, 64, "linear", 0.0), (1e4, 64, "linear", math.nan),
                 (1e4, 64, "base", math.inf), (1e4, 64, "by_parts", 8.0, 0.0, 1.0, 2.0),
                 (1e4, 64, "by_parts", 8.0, 1e4, 2.0, 2.0), (1e4, 64, "by_parts", 8.0, 1e4, -1.0, 2.0),
                 (1e4, 64, "by_parts", 8.0, 1e4, 1.0, math.inf), (1e4, 64, "by_parts", 8.0, 1e4, math.nan, 2.0)]:
        with pytest.raises(kvq.KvqError) as e:
            kvq.kvq_rope_table(*args)
        assert e.value.status == INVALID, args
    assert kvq.lib().kvq_rope_table(1e4, 64, None, None) == INVALID


def rope_struct(kvq, rot=128, layout=0, turns=64):
    s = kvq.KvqRope()
    s.rot_dim, s.layout, s.turns, s.scale = rot, layout, turns, 1.0
    return s


def heads_struct(kvq, x=256, out=4096, n=2, xt=256, xh=128, ot=256, oh=128):
    h = kvq.KvqHeads()
    h.x, h.out, h.num_heads = x, out, n
    h.x_token_stride, h.x_head_stride, h.out_token_stride, h.out_head_stride = xt, xh, ot, oh
    return h


def test_rope_apply_refusals(kvq):
    """Every refusal is taken on the host; the addresses are never read."""
    f = kvq.lib().kvq_rope_apply
    ref = ctypes.byref

    def call(rope=None, pos=64, a=None, b=None, t=3, d=128, tr=0):
        rope = rope if rope is not None else rope_struct(kvq)
        a = a if a is not None else heads_struct(kvq)
        return f(ref(rope), pos, ref(a), ref(b) if b is not None else None, t, d, tr, None)

    n = kvq.kvq_kernel_launches()
    assert call(t=0) == 0  # nothing to do
    assert f(None, 64, ref(heads_struct(kvq)), None, 3, 128, 0, None) == INVALID
    assert f(ref(rope_struct(kvq)), 64, None, None, 3, 128, 0, None) == INVALID
    for d in (0, 32, 96, 512):
        assert call(d=d) == UNSUPPORTED
    for bad in (dict(rot=0), dict(rot=3), dict(rot=130), dict(rot=-2), dict(layout=2), dict(layout=-1),
                dict(turns=0), dict(turns=68)):
        assert call(rope=rope_struct(kvq, **bad)) == INVALID, bad
    assert call(t=-1) == INVALID and call(pos=None) == INVALID and call(pos=66) == INVALID and call(tr=2) == INVALID
    for bad in (dict(x=0), dict(out=0), dict(x=257), dict(out=4097), dict(n=0), dict(xt=-1), dict(xh=-8), dict(ot=-1),
                dict(ot=200), dict(oh=64), dict(ot=0), dict(xt=1 << 40),
                dict(out=256, ot=512)):  # in place with other strides
        assert call(a=heads_struct(kvq, **bad)) == INVALID, bad
        assert call(b=heads_struct(kvq, **bad)) == INVALID, bad
    assert kvq.kvq_kernel_launches() == n


def test_rope_append_and_dequantize_refusals(kvq):
    ref = ctypes.byref
    d, hkv = 128, 2
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 4, "codebook", "int4_g32", 4, 0, signs, signs, device="cpu")

    def struct(**kw):
        s = kvq.KvqCache()
        ctypes.memmove(ref(s), ref(cache.struct), ctypes.sizeof(s))
        # addresses that are never read
        s.k_rows, s.v_rows, s.k_aux, s.v_aux, s.k_signs, s.v_signs = (1 << 12,) * 6
        for name, v in kw.items():
            setattr(s, name, v)
        return s

    def append(c=None, rope=None, pos=64, k=0, v=0, q=None, t=3, slots=64):
        k = heads_struct(kvq, out=None) if k == 0 else k
        v = heads_struct(kvq, out=None) if v == 0 else v
        return kvq.lib().kvq_rope_append(ref(c or struct()), ref(rope or rope_struct(kvq)), pos,
                                         ref(k) if k else None, ref(v) if v else None, ref(q) if q else None, t,
                                         slots, None)

    n = kvq.kvq_kernel_launches()
    assert append(t=0) == 0
    assert append(k=None, v=None) == INVALID
    assert append(pos=None) == INVALID and append(slots=None) == INVALID and append(slots=66) == INVALID
    assert append(t=-1) == INVALID
    assert append(rope=rope_struct(kvq, rot=256)) == INVALID
    for bad in (dict(x=264), dict(xt=260), dict(xh=132), dict(n=3), dict(x=0), dict(xt=-256)):
        assert append(k=heads_struct(kvq, **bad)) == INVALID, bad
        assert append(v=heads_struct(kvq, **bad)) == INVALID, bad
    assert append(q=heads_struct(kvq, out=0)) == INVALID
    assert append(c=struct(k_bounds=None)) == INVALID
    assert append(c=struct(k_signs=(1 << 12) + 8)) == INVALID
    assert append(c=struct(k_rows=None)) == INVALID
    assert append(c=struct(head_dim=96)) == UNSUPPORTED
    assert append(c=struct(v_format=4)) in (INVALID, UNSUPPORTED)  # a sketch on values
    assert append(t=(1 << 28) // hkv + 1) == INVALID

    def read(c=None, slots=64, t=3, k=256, v=256):
        return kvq.lib().kvq_dequantize(ref(c or struct()), slots, t, k, v, None)

    assert read(t=0) == 0
    assert read(k=None, v=None) == INVALID and read(slots=None) == INVALID and read(slots=65) == INVALID
    assert read(t=-1) == INVALID and read(k=264) == INVALID and read(v=258) == INVALID
    assert read(c=struct(v_signs=(1 << 12) + 4)) == INVALID
    assert read(c=struct(k_rows=8)) == INVALID
    assert read(c=struct(k_centroids=None)) == INVALID
    assert read(c=struct(num_pages=0)) == 0  # a pool without pages holds no slot
    assert kvq.lib().kvq_dequantize(None, 64, 3, 256, 256, None) == INVALID
    assert kvq.kvq_kernel_launches() == n


def test_binding_checks(kvq):
    d, hkv, hq, t = 128, 2, 4, 5
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 4, "codebook", "codebook", 4, 4, signs, signs, device="cpu").struct
    rope = kvq.Rope(128, "half", device="cpu")
    pos, slots = dev((t,), torch.int32), dev((t,), torch.int32)
    q, k = heads(t, hq, d), heads(t, hkv, d)
    with pytest.raises(AssertionError):  # valid: the call goes as far as the pointers
        kvq.kvq_rope_apply(rope, pos, q, k)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_rope_apply(rope, pos, torch.zeros((t, hq, d), dtype=torch.float16))
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_rope_apply(rope, pos, heads(t, hq * d))
    with pytest.raises(TypeError):
        kvq.kvq_rope_apply(rope, pos, heads(t, hq, d, dtype=torch.float32))
    with pytest.raises(TypeError):
        kvq.kvq_rope_apply(rope, dev((t,), torch.int64), q)
    with pytest.raises(ValueError, match="elements"):
        kvq.kvq_rope_apply(rope, dev((t - 1,), torch.int32), q)
    with pytest.raises(ValueError, match="adjacent"):
        kvq.kvq_rope_apply(rope, pos, Heads(torch.zeros((t, d, hq), dtype=torch.float16).transpose(1, 2)))
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_rope_apply(rope, pos, q, heads(t + 1, hkv, d))
    with pytest.raises((ValueError, AssertionError)):
        kvq.kvq_rope_apply(rope, pos, q, q_out=heads(t, hq + 1, d))
    with pytest.raises(ValueError, match="head"):
        kvq.kvq_rope_apply(rope, pos, heads(t, 0, d))

    with pytest.raises(AssertionError):
        kvq.kvq_rope_append(cache, rope, pos, k, k, slots, q)
    with pytest.raises(ValueError):
        kvq.kvq_rope_append(cache, rope, pos, None, None, slots, q)
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_rope_append(cache, rope, pos, heads(t, hkv + 1, d), None, slots)
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_rope_append(cache, rope, pos, k, heads(t - 1, hkv, d), slots)
    with pytest.raises(ValueError, match="elements"):
        kvq.kvq_rope_append(cache, rope, pos, k, k, dev((t - 1,), torch.int32))

    out = heads(t, hkv, d)
    with pytest.raises(AssertionError):
        kvq.kvq_dequantize(cache, slots, out, None)
    with pytest.raises(ValueError):
        kvq.kvq_dequantize(cache, slots)
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_dequantize(cache, slots, heads(t - 1, hkv, d))
    with pytest.raises(TypeError):
        kvq.kvq_dequantize(cache, slots, out, heads(t, hkv, d, dtype=torch.float32))


def shared_call(kvq, tiers, prefix, offsets, own, batch=4, hq=4, q=1 << 12, out=1 << 12, ws=1 << 12, ws_bytes=1 << 40,
                status=None, size=False):
    """kvq_decode_attention_shared (or its size function) on addresses that are never read."""
    def views(which):
        arr = (kvq.KvqTierView * max(1, len(which)))()
        for v, (c, table, lens, pages) in zip(arr, which):
            v.cache, v.block_table, v.seq_lens, v.max_pages = ctypes.pointer(c), table, lens, pages
        return arr
    off = (ctypes.c_int32 * len(offsets))(*offsets) if offsets is not None else None
    groups = len(offsets) - 1 if offsets is not None else 1
    if size:
        n = ctypes.c_size_t()
        st = kvq.lib().kvq_decode_shared_workspace_size(views(prefix), len(prefix), off, groups, views(own), len(own),
                                                        batch, hq, ctypes.byref(n))
        return st, n.value
    return kvq.lib().kvq_decode_attention_shared(views(prefix), len(prefix), off, groups, views(own), len(own), q,
                                                 batch, hq, out, ws, ws_bytes, status, None)


def test_shared_refusals(kvq):
    d, hkv = 128, 2
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 64, "codebook", "codebook", 4, 4, signs, signs, device="cpu")

    def struct(**kw):
        s = kvq.KvqCache()
        ctypes.memmove(ctypes.byref(s), ctypes.byref(cache.struct), ctypes.sizeof(s))
        s.k_rows, s.v_rows, s.k_aux, s.v_aux, s.k_signs, s.v_signs = (1 << 12,) * 6
        for name, v in kw.items():
            setattr(s, name, v)
        return s

    c = struct()
    view = (c, 64, 64, 8)
    ok = dict(tiers=None, prefix=[view], offsets=[0, 4], own=[view])
    st, need = shared_call(kvq, **ok, size=True)
    assert st == 0 and need > 0
    n = kvq.kvq_kernel_launches()
    assert shared_call(kvq, **ok, batch=0) == INVALID  # offsets beyond the batch
    assert shared_call(kvq, None, [view], [0, 0], [view], batch=0) == 0  # nothing to do
    for offsets in ([1, 0], [-1, 4], [0, 5], [0, 3, 2, 4], None, [0] * (kvq.MAX_PREFIX_GROUPS + 2)):
        assert shared_call(kvq, None, [view], offsets, [view]) == INVALID, offsets
        assert shared_call(kvq, None, [view], offsets, [view], size=True)[0] == INVALID, offsets
    assert shared_call(kvq, None, [], [0, 4], [view]) == INVALID  # no prefix tier
    assert shared_call(kvq, None, [view] * 3, [0, 4], [view] * 2) == INVALID  # five tiers
    for bad in ((c, 0, 64, 8), (c, 64, 0, 8), (c, 66, 64, 8), (c, 64, 65, 8), (c, 64, 64, -1)):
        assert shared_call(kvq, None, [bad], [0, 4], [view]) == INVALID, bad[1:]
        assert shared_call(kvq, None, [view], [0, 4], [bad]) == INVALID, bad[1:]
    for other in (struct(page_size=32), struct(num_kv_heads=4), struct(k_signs=1 << 13), struct(k_rows=0)):
        assert shared_call(kvq, None, [view], [0, 4], [(other, 64, 64, 8)]) == INVALID
    assert shared_call(kvq, **ok, hq=3) == INVALID and shared_call(kvq, **ok, hq=6) == UNSUPPORTED
    assert shared_call(kvq, **ok, hq=32) == UNSUPPORTED  # sixteen query heads per kv head
    for bad in (dict(q=0), dict(q=(1 << 12) + 8), dict(out=0), dict(out=(1 << 12) + 2), dict(ws=0),
                dict(ws=(1 << 12) + 128), dict(status=66)):
        assert shared_call(kvq, **ok, **bad) == INVALID, bad
    assert shared_call(kvq, **ok, ws_bytes=need - 1) == 3  # KVQ_ERR_WORKSPACE_TOO_SMALL
    assert shared_call(kvq, None, [view], [0, 4], [view], batch=(1 << 22) + 1) == UNSUPPORTED
    assert kvq.lib().kvq_decode_shared_workspace_size(None, 1, None, 1, None, 0, 4, 4, None) == INVALID
    assert kvq.kvq_kernel_launches() == n


def test_shared_binding_checks(kvq):
    d, hkv, hq, b = 128, 2, 4, 3
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 4, "codebook", "codebook", 4, 4, signs, signs, device="cpu")
    view = lambda rows, lens=None: kvq.TierView(cache, dev((rows, 4), torch.int32), dev((lens or rows,), torch.int32))  # noqa: E731
    q, out, ws = dev((b, hq, d), torch.float16), dev((b, hq, d), torch.float16), dev((64,), torch.uint8)
    call = kvq.kvq_decode_attention_shared
    with pytest.raises(AssertionError):  # valid: as far as the pointers
        call([view(1)], [0, 3], [view(b)], q, out, ws)
    with pytest.raises(AssertionError):
        call([view(2)], [0, 1, 3], None, q, out, ws)
    with pytest.raises(TypeError):
        call([view(1)], [0, 3], [view(b)], q, dev((b, hq, d), torch.float32), ws)
    with pytest.raises(ValueError, match="shape"):
        call([view(1)], [0, 3], [view(b)], dev((b, hq, 64), torch.float16), out, ws)
    with pytest.raises(ValueError, match="tier"):
        call([], [0, 3], [view(b)], q, out, ws)
    with pytest.raises(ValueError, match="group_offsets"):
        call([view(1)], [0], [view(b)], q, out, ws)
    with pytest.raises(ValueError, match="rows"):
        call([view(1, 2)], [0, 1, 3], [view(b)], q, out, ws)
    with pytest.raises(ValueError, match="elements"):
        call([view(1)], [0, 3], [view(b, b - 1)], q, out, ws)
    with pytest.raises(ValueError, match="workspace"):
        call([view(1)], [0, 3], [view(b)], q, out, None)
    with pytest.raises(TypeError):
        call([view(1)], [0, 3], [view(b)], q, out, ws, status=dev((1,), torch.int64))


def test_shared_prefix_tables_stay_inside_32_bits(kvq):
    """A table that names pages again and again may reach 2^31 tokens from a small pool.  The prefix
    pass counts tokens in 32 bits up to the end of the last tile: a table whose last tile may end
    beyond is refused, whatever the kernel family, before anything is launched."""
    d, hkv = 128, 2
    signs = np.ones((hkv, d), dtype=np.int8)
    n = kvq.kvq_kernel_launches()
    for fmt, bits in (("codebook", 4), ("fp16", 0)):
        cache = kvq.PagedCache(d, hkv, 2, fmt, fmt, bits, bits, signs, signs, page_size=16, device="cpu")

        def struct(ps):
            s = kvq.KvqCache()
            ctypes.memmove(ctypes.byref(s), ctypes.byref(cache.struct), ctypes.sizeof(s))
            s.k_rows, s.v_rows, s.k_signs, s.v_signs = (1 << 12,) * 4
            s.k_aux = s.v_aux = 1 << 12
            s.page_size = ps
            return s

        for ps, most in ((16, (1 << 27) - 17), (1 << 20, (1 << 11) - 1)):
            c = struct(ps)
            assert shared_call(kvq, None, [(c, 64, 64, most)], [0, 4], [], size=True)[0] == 0, ps
            for pages in (most + 1, 1 << 30):
                assert shared_call(kvq, None, [(c, 64, 64, pages)], [0, 4], [], size=True)[0] == UNSUPPORTED, (ps, pages)
                assert shared_call(kvq, None, [(c, 64, 64, pages)], [0, 4], []) == UNSUPPORTED, (ps, pages)
                if ps > 16:  # a tier behind a shorter one
                    both = [(c, 64, 64, 1), (c, 64, 64, pages)]
                    assert shared_call(kvq, None, both, [0, 4], []) == UNSUPPORTED
    assert kvq.kvq_kernel_launches() == n


class On(Heads):
    """A stand-in on a device, with an address that is never read."""

    def __init__(self, t, index=0):
        super().__init__(t)
        self.index = index

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 12

    def element_size(self):
        return self.t.element_size()


class Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 77


def test_serving_calls_stay_on_the_current_device(kvq, monkeypatch):
    """The library launches on the current device: tensors of another one, a stream of another one and
    tensors of two are refused by the binding, whether the caller names a stream or not."""
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or 0

    d, hkv, hq, t = 128, 2, 4, 3
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 4, "codebook", "codebook", 4, 4, signs, signs, device="cpu")
    rope = kvq.Rope(128, "half", device="cpu")
    monkeypatch.setattr(kvq, "_lib_handle", Library())
    monkeypatch.setattr(kvq, "_current_device", lambda: 0)
    monkeypatch.setattr(kvq, "_raw_stream", lambda index: 1000 + index)
    on = lambda shape, dtype=torch.float16, index=0: On(torch.zeros(shape, dtype=dtype), index)  # noqa: E731
    i32 = torch.int32

    def calls(index, stream, odd=None):
        """The four calls with tensors on `index`, one of them (odd) on the other device."""
        at = lambda name: 1 - index if name == odd else index  # noqa: E731
        rope.turns = On(torch.zeros(64, dtype=torch.int64), at("turns"))
        pos, slots = on((t,), i32, at("ints")), on((t,), i32, index)
        q, k = on((t, hq, d), index=index), on((t, hkv, d), index=at("heads"))
        view = lambda n: kvq.TierView(cache, on((n, 4), i32, at("table")), on((n,), i32, index))  # noqa: E731
        yield "turns ints heads", lambda: kvq.kvq_rope_apply(rope, pos, q, k, stream=stream)
        yield "turns ints heads", lambda: kvq.kvq_rope_append(cache.struct, rope, pos, k, k, slots, q, stream=stream)
        yield "ints heads", lambda: kvq.kvq_dequantize(cache.struct, pos, k, on((t, hkv, d), index=index), stream=stream)
        yield "table", lambda: kvq.kvq_decode_attention_shared([view(1)], [0, t], [view(t)], q, on((t, hq, d), index=index),
                                                               on((64,), torch.uint8, index), stream=stream)

    for stream, handle in ((None, 1000), (0, 0), (5, 5), (Stream(0), 77)):
        for _, call in calls(0, stream):
            call()
            assert seen.pop()[1][-1] == handle and not seen  # the stream is every call's last argument
    for stream in (None, 0, 5, Stream(0), Stream(1)):
        for _, call in calls(1, stream):
            with pytest.raises(ValueError, match="device"):
                call()
        for odd in ("turns", "ints", "heads", "table"):
            for parts, call in calls(0, stream, odd):
                if odd in parts:
                    with pytest.raises(ValueError, match="device"):
                        call()
    for _, call in calls(0, Stream(1)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not seen


def test_misaligned_int4_scales_leave_the_fused_kernel(kvq):
    """The fused fp16 / fp8 kernel copies INT4 scales 16 bytes at a time: scales at other addresses make
    the plan of the generic kernel (as another alignment of the signs does), in the plain and in the
    shared decode."""
    d, hkv, hq, b = 128, 2, 8, 4
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 64, "fp8_e4m3", "int4_g32", 0, 0, signs, signs, device="cpu")

    def struct(**kw):
        s = kvq.KvqCache()
        ctypes.memmove(ctypes.byref(s), ctypes.byref(cache.struct), ctypes.sizeof(s))
        s.k_rows, s.v_rows, s.k_aux, s.v_aux, s.k_signs, s.v_signs = (1 << 12,) * 6
        for name, v in kw.items():
            setattr(s, name, v)
        return s

    def plain(c):
        arr = (kvq.KvqTierView * 1)()
        arr[0].cache, arr[0].block_table, arr[0].seq_lens, arr[0].max_pages = ctypes.pointer(c), 64, 64, 512
        n = ctypes.c_size_t()
        assert kvq.lib().kvq_decode_workspace_size(arr, 1, b, hq, 0, ctypes.byref(n)) == 0
        return n.value

    def shared(c):
        view = (c, 64, 64, 512)
        st, n = shared_call(kvq, None, [view], [0, b], [view], batch=b, hq=hq, size=True)
        assert st == 0
        return n

    generic = struct(k_signs=(1 << 12) + 4, v_signs=(1 << 12) + 4)
    for off in (2, 4, 8, 14):
        bad = struct(v_aux=(1 << 12) + off)
        # (the size covers queries at any address, the generic kernel's plan too: never the smaller one)
        assert plain(bad) == plain(generic)
        if off % 8:
            assert shared(bad) == shared(generic)
    assert shared(struct(v_aux=(1 << 12) + 8)) != shared(struct())  # own tiers: another kernel's chunks
    assert plain(struct()) >= plain(generic)


def test_append_refuses_signs_it_cannot_read(kvq):
    """A lane reads the signs of head_dim / 32 coordinates at once: other addresses are refused before
    anything is launched, for the side that is appended."""
    for d in (64, 128, 256):
        signs = np.ones((2, d), dtype=np.int8)
        cache = kvq.PagedCache(d, 2, 4, "fp16", "fp16", 0, 0, signs, signs, device="cpu")
        s = kvq.KvqCache()
        ctypes.memmove(ctypes.byref(s), ctypes.byref(cache.struct), ctypes.sizeof(s))
        s.k_rows = s.v_rows = 1 << 12
        f = kvq.lib().kvq_quantize_append
        n = kvq.kvq_kernel_launches()
        for off in range(1, d // 32):
            s.k_signs, s.v_signs = (1 << 12) + off, 1 << 12
            assert f(ctypes.byref(s), 256, 256, 3, 64, None) == INVALID
            assert f(ctypes.byref(s), 256, None, 3, 64, None) == INVALID
            s.k_signs, s.v_signs = 1 << 12, (1 << 12) + off
            assert f(ctypes.byref(s), 256, 256, 3, 64, None) == INVALID
            assert f(ctypes.byref(s), None, 256, 3, 64, None) == INVALID
        assert kvq.kvq_kernel_launches() == n
