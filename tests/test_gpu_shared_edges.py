"""kvq_decode_attention_shared where the prefix pass leaves its usual course: running maxima that are
raised again and again, pages outside the pool, values at the ends of their formats.

u = 2^-11 (half a step of fp16).  Expectations are attention in float64 over what the cache holds,
read back by kvq_dequantize (rounded once more, u of a vector) or decoded by the oracle."""
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import cache as ocache
from oracle import shared as oshared
from tests import gpu_util as gu
from tests.test_gpu_shared import SPECS, Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


def modules():
    return gu.torch_cuda(), gu.kvq_module()


def call(kvq, torch, prefix, offsets, own, q, status=0):
    """The shared decode of q (numpy fp16 [B, Hq, D]) as float64."""
    qd = torch.from_numpy(np.ascontiguousarray(q)).cuda()
    out = torch.empty_like(qd)
    need = kvq.kvq_decode_shared_workspace_size(prefix, offsets, own, q.shape[0], q.shape[1])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    bits = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    kvq.kvq_decode_attention_shared(prefix, offsets, own, qd, out, ws, bits)
    assert int(bits.item()) == status
    return out.cpu().numpy().astype(np.float64)


def read_back(kvq, torch, cache, tokens):
    hkv, d = cache.num_kv_heads, cache.head_dim
    k, v = (torch.empty(tokens, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    kvq.kvq_dequantize(cache.struct, torch.arange(tokens, dtype=torch.int32, device="cuda"), k, v)
    return k.cpu().numpy().astype(np.float64), v.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("batch", [2, 20])  # 16 rows: tiles in turn between the softmax groups; 160: every tile both
@pytest.mark.parametrize("fmt,bits", [("fp16", 0), ("codebook", 4)])
def test_maxima_that_rise_in_both_halves_of_a_tile(fmt, bits, batch):
    """Four tiles of one work item (320 kv heads leave one chunk): scores level in the first two, then
    2^9 and 2^18 times the weight in the halves of the third and of the fourth.  Whichever tiles a softmax group takes,
    its second one raises the maximum twice: the accumulator is rescaled, and rescaled again with
    the half's weights that were just stored.  The level tiles' values are 64 times one vector: beside
    the mean of 128 vectors (2-norm 1) they count 256 2^-18 / 128 64 sqrt(128) = 2^-7.5, and with one
    of the two rescalings lost 2^9 times that.

    Tolerance (2-norm): a half's weights are alike and so is their rounding (u), values, output and
    read-back are rounded (u each), together at most 4 u = 2^-9; a score (at most 12.5 nats) is off
    by u sqrt(3) of itself at most, 0.011, which moves the shares of the lighter levels (2^-8 and 2^-7.5) by as
    much of themselves."""
    torch, kvq = modules()
    d, ps, hkv, group, n = 128, 16, 320, 8, 512
    rng = np.random.default_rng(bits + batch)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    cache = kvq.PagedCache(d, hkv, n // ps, fmt, fmt, bits, bits, ks, vs, ps)
    level = np.zeros(n)
    level[256:320], level[320:384], level[384:448], level[448:] = 9.0, 18.0, 9.0, 18.0
    u = rng.standard_normal((hkv, d))
    u /= np.linalg.norm(u, axis=-1, keepdims=True)
    length = 12.0  # of a query; a key of length x scores length x / sqrt(d) nats
    x = (level * math.log(2.0) + 0.5) * math.sqrt(d) / length  # (half a nat: no key is zero)
    k = (x[:, None, None] * u).astype(np.float16)
    v = rng.standard_normal((n, hkv, d))
    v[:256] = 64 * v[0]
    cache.append(torch.from_numpy(k).cuda(), torch.from_numpy(v.astype(np.float16)).cuda(),
                 torch.arange(n, dtype=torch.int32, device="cuda"))
    view = kvq.TierView(cache, torch.arange(n // ps, dtype=torch.int32, device="cuda")[None],
                        torch.tensor([n], dtype=torch.int32, device="cuda"))
    q = np.repeat((length * u).astype(np.float16), group, 0)[None].repeat(batch, 0)
    got = call(kvq, torch, [view], [0, batch], None, q)
    kb, vb = read_back(kvq, torch, cache, n)
    for h in range(0, hkv, 13):
        s = kb[:, h] @ q[0, h * group].astype(np.float64) / math.sqrt(d)
        p = np.exp(s - s.max())
        want = (p / p.sum()) @ vb[:, h]
        limit = 2.0 ** -9 * np.linalg.norm(want) + 0.011 * (2.0 ** -8 + 2.0 ** -7.5)
        for b in (0, batch - 1):
            assert np.all(np.linalg.norm(got[b, h * group:(h + 1) * group] - want, axis=-1) <= limit)


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "cb4", "cb32"])
@pytest.mark.parametrize("length", [100, 128, 900])
@pytest.mark.parametrize("batch,group", [(3, 2), (40, 4)])
def test_a_page_outside_the_pool_is_left_out(name, length, batch, group):
    """The chunk of the prefix that holds the page counts for nothing: one tile is one chunk, and a
    longer prefix loses a run of whole tiles around the page, whatever the plan made of it.  Other
    groups keep theirs."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[length, 70]], [0, batch, batch + 2], [name], [[5] * (batch + 2)], hq=2 * group, hkv=2,
             seed=length + batch)
    rows = [b for b in (0, 1, batch - 1)]
    heads = {(b, h) for b in rows for h in (0, 2 * group - 1)}
    other = {(b, h) for b in (batch, batch + 1) for h in (0, 2 * group - 1)}
    tiles = -(-length // 128)
    keep = c.prefix[0].block_table.clone()
    for at in sorted({0, tiles // 2, tiles - 1}):  # the page's tile
        for bad in (-1, c.built.gpu[0].num_pages):
            c.prefix[0].block_table.copy_(keep)
            c.prefix[0].block_table[0, min(8 * at + 2, (length - 1) // 16)] = bad
            got = call(kvq, torch, c.prefix, c.offsets, c.own, c.q, kvq.DEVERR_PAGE_INDEX)
            c.check(got, other)
            want = {}
            for per in range(1, tiles + 1):  # tiles of a chunk
                lo = at // per * per
                want[lo, min(lo + per, tiles)] = None
            fits = []
            for lo, hi in want:
                try:
                    check_without(c, got, heads, lo * 128, min(hi * 128, length))
                    fits.append((lo, hi))
                except AssertionError:
                    pass
            assert fits, "the output fits no chunk left out"
            if tiles == 1:
                assert fits == [(0, 1)]


def check_without(c, got, heads, lo, hi):
    """The output against attention without tokens [lo, hi) of group 0's prefix (2-norm, 2^-9 of the
    output as in test_gpu_shared)."""
    grp = c.hq // c.hkv
    off = size = 0.0
    for b, h in heads:
        keys, values = oatt.dequantised_kv(c.tiers, b, h // grp)
        n = int(c.tiers[0].lens[b])
        there = np.r_[0:lo, hi:n, n:len(keys)]
        s = keys[there] @ c.q[b, h].astype(np.float64) / math.sqrt(c.d)
        w = np.exp(s - s.max())
        want = (w / w.sum()) @ values[there]
        off += float(np.sum((got[b, h] - want) ** 2))
        size += float(np.sum(want ** 2))
    assert math.sqrt(off / size) <= 2.0 ** -9, math.sqrt(off / size)


def check_norm(c, got, heads, limit):
    off = size = 0.0
    for b, h in heads:
        keys, values = oatt.dequantised_kv(c.tiers, b, h // (c.hq // c.hkv))
        s = keys @ c.q[b, h].astype(np.float64) / math.sqrt(c.d)
        w = np.exp(s - s.max())
        want = (w / w.sum()) @ values
        off += float(np.sum((got[b, h] - want) ** 2))
        size += float(np.sum(want ** 2))
    assert math.sqrt(off / size) <= limit, math.sqrt(off / size)


def put_large_values(torch, c, side, sequences, size):
    """Every third value of a tier along the signs, so that one rotated coordinate holds it all: in the
    oracle's pool and in the cache."""
    tier, cache = c.built.ora[side], c.built.gpu[side]
    ps = tier.page_size
    for i in range(sequences):
        t = np.arange(0, int(tier.lens[i]), 3)
        v = (np.where((i + t) % 2, 1.0, 0.4) * size)[:, None, None] * c.built.v_signs
        ocache.write(tier.v, tier.block_table[i][t // ps] * ps + t % ps, v.astype(np.float16), ps)
    cache.v_rows.copy_(torch.from_numpy(tier.v.rows))
    cache.v_aux.copy_(torch.from_numpy(tier.v.aux.reshape(cache.v_aux.shape)))


@pytest.mark.parametrize("size", [100.0, 157.0, 160.0, 1000.0, 25000.0])
@pytest.mark.parametrize("batch,group", [(3, 2), (4, 8)])
def test_int4_scales_of_any_size_in_the_sequences_own_tier(size, batch, group):
    """Scales (1.6 times the size) up to 2^8 and beyond, whose product with a weight times 2^8 passes fp16's
    largest number: by kvq_decode_attention too, whose weights keep 22 bits (2^-16 with the
    scores' float32 errors)."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[200]], [0, batch], ["fp8_int4"], [[300, 21, 16, 5][:batch]], hq=2 * group, hkv=2,
             seed=int(size))
    put_large_values(torch, c, 1, batch, size)
    assert np.max(c.tiers[1].v.aux.astype(np.float64)) > 1.5 * size
    heads = {(b, h) for b in range(batch) for h in range(2 * group)}
    check_norm(c, call(kvq, torch, c.prefix, c.offsets, c.own, c.q), heads, 2.0 ** -9)
    own = gu.gpu_decode(kvq, torch, c.own, c.q).astype(np.float64)
    c.tiers = c.tiers[1:]
    check_norm(c, own, heads, 2.0 ** -16)


@pytest.mark.parametrize("size", [157.0, 160.0, 5700.0, 5900.0, 25000.0])
@pytest.mark.parametrize("batch,group", [(3, 2), (40, 4)])
def test_int4_scales_of_a_prefix(size, batch, group):
    """Scales whose values fit fp16 (up to 9352) are attended, larger ones are reported."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[400]], [0, batch], ["fp8_int4"], [[7] * batch], hq=2 * group, hkv=2,
             seed=int(size))
    put_large_values(torch, c, 0, 1, size)
    most = np.max(c.tiers[0].v.aux.astype(np.float64))
    assert (most > 9352) == (size > 5800)
    got = call(kvq, torch, c.prefix, c.offsets, c.own, c.q, kvq.DEVERR_VALUE_RANGE if most > 9352 else 0)
    if most <= 9352:
        check_norm(c, got, {(b, h) for b in (0, 1, batch - 1) for h in range(2 * group)}, 2.0 ** -9)


@pytest.mark.parametrize("name,d,hq", [("fp16", 128, 8), ("fp8_int4", 128, 8), ("cb4", 128, 8), ("cb4", 128, 2),
                                       ("cb32", 128, 4), ("fp8_fp16", 128, 8), ("fp16", 64, 4), ("fp8_int4", 256, 4),
                                       ("cb4", 256, 2), ("qjl", 128, 4), ("outlier", 128, 4)])
def test_what_lies_behind_the_sequences_is_not_attended(name, d, hq):
    """NaN in every slot of the pool that holds no token, those behind a sequence's last token in its
    last page among them: the outputs of the shared and of the plain decode stay the same, to the bit."""
    torch, kvq = modules()
    lens = [1, 15, 16, 17, 250, 0]
    c = Case(kvq, torch, ["fp8_int4" if name in ("qjl", "outlier") else name], [[40]], [0, 6], [name], [lens], hq=hq, hkv=2,
             d=d, seed=d + hq)
    run = lambda: (call(kvq, torch, c.prefix, c.offsets, c.own, c.q), gu.gpu_decode(kvq, torch, c.own, c.q))  # noqa: E731
    want = run()
    assert all(np.isfinite(x).all() for x in want)
    cache, table = c.built.gpu[1], c.own[0].block_table.cpu().numpy()
    held = np.concatenate([table[i][np.arange(n) // 16] * 16 + np.arange(n) % 16 for i, n in enumerate(lens)])
    free = np.setdiff1d(np.arange(cache.num_pages * 16), held)
    pages, offs = (torch.from_numpy(x).cuda() for x in (free // 16, free % 16))
    for a in (cache.k_rows, cache.v_rows, cache.k_aux, cache.v_aux):
        if a is not None and a.dtype == torch.float16:
            a[pages, :, offs] = float("nan")
        elif a is not None:  # bytes of NaN in fp16 and in fp8 rows, of -1 and a NaN norm in codes and outliers
            a[pages, :, offs] = 0x7F if a is cache.k_aux or "fp" in name else 0xFF
    for got, x in zip(run(), want):
        assert np.array_equal(got, x)


@pytest.mark.parametrize("name,d,hq", [("fp16", 128, 8), ("fp8_int4", 128, 8), ("cb4", 128, 8), ("cb4", 128, 2),
                                       ("cb32", 128, 4), ("fp8_fp16", 128, 8), ("fp16", 64, 4), ("fp8_int4", 256, 4),
                                       ("cb4", 256, 2)])
def test_a_query_that_is_not_finite_without_a_prefix(name, d, hq):
    """Sequences outside every group, of one token and of many, and one without any: a query with a NaN
    or an infinity gives NaN, of the shared and of the plain decode, and zeros only where no token is."""
    torch, kvq = modules()
    lens = [1, 40, 700, 0, 9]
    c = Case(kvq, torch, [name], [[30]], [4, 5], [name], [lens], hq=hq, hkv=2, d=d, seed=d + hq)
    want = call(kvq, torch, c.prefix, c.offsets, c.own, c.q), gu.gpu_decode(kvq, torch, c.own, c.q)
    keep = c.q.copy()
    bad = [(0, 0), (1, hq - 1), (2, 1), (3, 0), (4, hq - 1)]
    for i, (b, h) in enumerate(bad):
        c.q[b, h, 7] = (np.nan, np.inf, -np.inf, np.nan, np.nan)[i]
    got = call(kvq, torch, c.prefix, c.offsets, c.own, c.q), gu.gpu_decode(kvq, torch, c.own, c.q)
    c.q = keep
    for x, y in zip(got, want):
        for b, h in bad:
            if lens[b]:
                assert np.isnan(x[b, h]).all(), (b, h)
            x[b, h] = y[b, h] if lens[b] else x[b, h]
        assert np.array_equal(x, y)


@pytest.mark.parametrize("shift", [1, 4])  # fp16 numbers: 2 bytes, and the 8 that the prefix pass takes
def test_int4_scales_at_other_addresses(shift):
    """Scales that are not 16-byte aligned, of the prefix and of the sequences' own tier."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[300]], [0, 3], ["fp8_int4"], [[20, 0, 133]], hq=8, hkv=2, seed=shift)
    want = call(kvq, torch, c.prefix, c.offsets, c.own, c.q), gu.gpu_decode(kvq, torch, c.own, c.q)
    for cache in c.built.gpu:
        flat = torch.empty(cache.v_aux.numel() + 8, dtype=torch.float16, device="cuda")
        moved = flat[shift:shift + cache.v_aux.numel()].view(cache.v_aux.shape)
        moved.copy_(cache.v_aux)
        assert moved.data_ptr() % 16 == 2 * shift
        cache.v_aux, cache.struct.v_aux = moved, moved.data_ptr()
    c.check(call(kvq, torch, c.prefix, c.offsets, c.own, c.q))
    got = gu.gpu_decode(kvq, torch, c.own, c.q)
    assert np.linalg.norm(got - want[1]) <= 2.0 ** -16 * np.linalg.norm(want[1])


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "cb4", "cb32"])
def test_long_sequences_beside_a_prefix(name):
    """Sequences of their own long enough for hundreds of partial results a row, beside one of a few
    tokens and one of none: the joining pass goes over its partials more than once."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[3000]], [0, 3], [name], [[60000, 0, 77]], hq=4, hkv=1, seed=40)
    got = call(kvq, torch, c.prefix, c.offsets, c.own, c.q)
    c.check(got)


@pytest.mark.parametrize("name,d", [("fp16", 128), ("cb4", 128), ("fp16", 64)])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("offsets", [[0, 0], [2, 2, 2], [3, 3], [0, 2]])
def test_groups_without_sequences(offsets, own, name, d):
    """Groups without a sequence, eager and replayed: no prefix pass runs, sequences outside have their
    own tokens or none (zeros)."""
    torch, kvq = modules()
    lens = [[5, 0, 40]] if own else []
    c = Case(kvq, torch, [name], [[50] * (len(offsets) - 1)], offsets, [name] if own else [], lens or [[0] * 3], hq=4,
             hkv=2, d=d, seed=41)
    c.batch = 3
    c.q = np.random.default_rng(3).standard_normal((3, 4, d)).astype(np.float16)
    ora = c.built.ora
    c.tiers = oshared.as_tiers(ora[:1], offsets, ora[1:], 3)
    q = torch.from_numpy(c.q).cuda()
    out, again = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    ws = torch.full((kvq.kvq_decode_shared_workspace_size(c.prefix, offsets, c.own, 3, 4),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    bits = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    run = lambda to: kvq.kvq_decode_attention_shared(c.prefix, offsets, c.own, q, to, ws, bits)  # noqa: E731
    run(out)
    torch.cuda.synchronize()
    c.check(out.cpu().numpy())
    assert int(bits.item()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(again)
    ws.fill_(0xFF)
    bits.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and int(bits.item()) == 0


@pytest.mark.parametrize("name,d", [("fp8_int4", 128), ("cb4", 128), ("cb4", 256)])
def test_output_over_the_queries(name, d):
    """out may be q itself: every pass has read the queries before the last one writes."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[700]], [0, 20], [name], [[30] * 20], hq=8, hkv=2, d=d, seed=42)
    want = call(kvq, torch, c.prefix, c.offsets, c.own, c.q)
    q = torch.from_numpy(c.q).cuda()
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size(c.prefix, c.offsets, c.own, 20, 8), dtype=torch.uint8, device="cuda")
    kvq.kvq_decode_attention_shared(c.prefix, c.offsets, c.own, q, q, ws)
    assert np.array_equal(q.cpu().numpy().astype(np.float64), want)


def test_calls_on_many_streams_at_once():
    """Sixteen calls in flight on as many streams, of both kinds of prefix and several shapes, with a
    workspace each: the results of the calls alone."""
    torch, kvq = modules()
    cases = [Case(kvq, torch, [name], [[length]], [0, batch], [name], [[9] * batch], hq=8, hkv=2, seed=43 + i)
             for i, (name, length, batch) in enumerate([("cb4", 900, 6), ("fp8_int4", 3000, 40), ("fp16", 130, 2),
                                                        ("cb32", 5000, 33)])]
    q = [torch.from_numpy(c.q).cuda() for c in cases]
    want = [call(kvq, torch, c.prefix, c.offsets, c.own, c.q) for c in cases]
    jobs = []
    for i in range(16):
        c, x = cases[i % 4], q[i % 4]
        need = kvq.kvq_decode_shared_workspace_size(c.prefix, c.offsets, c.own, c.batch, 8)
        jobs.append((c, x, torch.empty_like(x), torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, x, out, ws, stream in jobs:
            kvq.kvq_decode_attention_shared(c.prefix, c.offsets, c.own, x, out, ws, stream=stream)
    torch.cuda.synchronize()
    for i, (_, _, out, _, _) in enumerate(jobs):
        assert np.array_equal(out.cpu().numpy().astype(np.float64), want[i % 4]), i


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "fp8_fp16", "cb4", "cb32", "cb23"])
@pytest.mark.parametrize("batch,group", [(2, 1), (8, 4), (33, 4)])
def test_error_beside_the_outputs_own_rounding(name, batch, group):
    """Keys and values with x30 outlier channels, as a model's: scores of several nats, a few tokens with
    most of the weight.  The output is rounded to fp16: 0.42 u of it (2-norm; u times the root mean square
    of a rounding over a binade, 1 / sqrt(3) 0.72).  Beside it stand one rounding each of the weights and of
    INT4 values (0.42 u) and of centroids (0.35 u of a key's score, which with several nats is as much of the
    output): 0.84 u in squares.  At most u.  A query rounded to one fp16 number alone would add
    0.5 to 1.3 u."""
    torch, kvq = modules()
    hkv, d, n = 8, 128, 2500
    rng = np.random.default_rng([batch, len(name)])
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    loud = lambda: np.where(rng.random((hkv, d)) < 0.015, 30.0, 1.0)  # noqa: E731
    draw = lambda L, f: (rng.standard_normal((L, hkv, d)) * f).astype(np.float16)  # noqa: E731
    fk, fv = loud(), loud()
    kv = [[(draw(n, fk), draw(n, fv))] + [(draw(0, fk), draw(0, fv))] * (batch - 1),
          [(draw(5, fk), draw(5, fv)) for _ in range(batch)]]
    built = gu.build_exact(kvq, torch, [SPECS[name], SPECS[name]], kv, ks, vs, 16, shuffle_seed=batch)
    first, second = (c.struct for c in built.gpu)
    second.k_signs, second.v_signs = first.k_signs, first.v_signs
    q = rng.standard_normal((batch, hkv * group, d)).astype(np.float16)
    got = call(kvq, torch, built.views[:1], [0, batch], built.views[1:], q)
    tiers = oshared.as_tiers(built.ora[:1], [0, batch], built.ora[1:], batch)
    off = size = 0.0
    for b in sorted({0, 1, batch // 2, batch - 1}):
        for h in range(hkv):
            keys, values = oatt.dequantised_kv(tiers, b, h)
            s = q[b, h * group:(h + 1) * group].astype(np.float64) @ keys.T / math.sqrt(d)
            w = np.exp(s - s.max(-1, keepdims=True))
            want = (w / w.sum(-1, keepdims=True)) @ values
            off += float(np.sum((got[b, h * group:(h + 1) * group] - want) ** 2))
            size += float(np.sum(want ** 2))
    assert math.sqrt(off / size) <= U, math.sqrt(off / size) / U


@pytest.mark.parametrize("how", ["any", "small first", "large first", "none first", "sink"])
@pytest.mark.parametrize("name", ["cb4", "cb32"])
@pytest.mark.parametrize("batch,group", [(2, 2), (12, 8)])
def test_values_of_any_norm(name, how, batch, group):
    """The prefix pass multiplies weights by the values' norms, over that of the item's first tile: norms
    from 2^-8 to 2^12 at random; a first tile 2^-14 or 2^14 times the others; a first tile of zeros; a
    token of value zero that outweighs all others 2^30 times (what is left of the output is tiny, and
    fp16's smallest step, 2^-25 of a weight of 2, of every token bounds it)."""
    torch, kvq = modules()
    hkv, d, n = 4, 128, 1500
    rng = np.random.default_rng([batch, len(how), len(name)])
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    size = np.ones(n)
    if how == "any":
        size = 2.0 ** rng.uniform(-11, 9, n)
    elif how != "sink":
        size[:128] = {"small first": 2.0 ** -14, "large first": 2.0 ** 12, "none first": 0.0}[how]
        size[128:] = {"small first": 1.0, "large first": 0.25, "none first": 1.0}[how]
    k = (0.3 * rng.standard_normal((n, hkv, d))).astype(np.float16)
    v = rng.standard_normal((n, hkv, d)) * size[:, None, None]
    q = rng.standard_normal((batch, hkv, d)).repeat(group, 1)
    if how == "sink":
        q[:] = q[0]
        u = q[0, ::group] / np.linalg.norm(q[0, ::group], axis=-1, keepdims=True)
        k[5] = 30 * math.log(2.0) * math.sqrt(d) / np.linalg.norm(q[0, ::group], axis=-1, keepdims=True) * u
        v[5] = 0
    empty = np.zeros((0, hkv, d), np.float16)
    kv = [[(k, v.astype(np.float16))] + [(empty, empty)] * (batch - 1)]
    built = gu.build_exact(kvq, torch, [SPECS[name]], kv, ks, vs, 16, shuffle_seed=batch)
    q = q.astype(np.float16)
    got = call(kvq, torch, built.views, [0, batch], None, q)
    tiers = oshared.as_tiers(built.ora, [0, batch], [], batch)
    for b in sorted({0, batch - 1}):
        for h in range(hkv):
            keys, values = oatt.dequantised_kv(tiers, b, h)
            s = q[b, h * group:(h + 1) * group].astype(np.float64) @ keys.T / math.sqrt(d)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            want = w @ values
            off = np.linalg.norm(got[b, h * group:(h + 1) * group] - want, axis=-1)
            floor = 2.0 ** -25 * math.sqrt(d)  # fp16 outputs below its normal numbers
            if how == "sink":
                floor += 2.0 ** -25 * np.linalg.norm(values, axis=-1).max() * math.sqrt(n)
            assert np.all(off <= 2.0 ** -9 * np.linalg.norm(want, axis=-1) + floor), (off, np.linalg.norm(want, axis=-1))
