"""GPU parity of kvq_rope_append: queries against the rotary oracle, stored rows against the
oracle's encode of the turned keys.

Tolerance, derived before the first run.  A turned float32 element is within (|a| + |b|) s
2^-21 of the exact one (tests/test_gpu_rope.py); a rotated coordinate then within
  tau = s (2 sum|x|) / sqrt(D) (2^-21 + (log2 D + 2) 2^-24),
since sum(|a| + |b|) over the elements is 2 sum|x| and the turned elements' sum is no larger
than s times that.  What is stored is monotone in the coordinate, so it must lie between what
the oracle stores for x~ - tau and x~ + tau: for codes, u = sqrt(D) x~ / ||x~|| moves by
sqrt(D) tau / n, and with the norm's own error (tau sqrt(D) / n relative, and 2^-22 for the
float32 sum) by |u| times that; the fp16 norm is the rounding of a value that close; INT4
scales and levels likewise."""
import math

import numpy as np
import pytest

from oracle import cache as ocache
from oracle import formats as ofmt
from oracle import rope as orope
from oracle import rotation as orot
from tests import gpu_util as gu
from tests.test_gpu_rope import check as check_rope, frequencies, make_rope

pytestmark = pytest.mark.gpu

FORMATS = [("codebook", 4, "codebook", 4), ("codebook", 3, "codebook", 2), ("codebook", 2, "codebook", 3),
           ("fp16", 0, "fp16", 0), ("fp8_e4m3", 0, "int4_g32", 0), ("int4_g32", 0, "fp8_e4m3", 0)]


def check_side(xr, tau, fmt, bits, rows, aux):
    """xr [T, d] exact rotated vectors, tau [T, 1]."""
    d = xr.shape[-1]
    if fmt == "codebook":
        n = np.sqrt(np.sum(xr * xr, -1, keepdims=True))
        assert np.all(n > 0)
        u = math.sqrt(d) * xr / n
        rel = math.sqrt(d) * tau / n + 2.0 ** -22
        du = (math.sqrt(d) * tau / n + np.abs(u) * rel) * (1 + 2.0 ** -9)
        b32 = gu.tables("lloyd_max", bits)[1].astype(np.float64)
        lo = np.sum((u - du)[..., None] > b32, -1)
        hi = np.sum((u + du)[..., None] > b32, -1)
        idx = ofmt.unpack_bits(rows, bits, d)
        assert np.all((idx >= lo) & (idx <= hi)), f"{int(np.sum((idx < lo) | (idx > hi)))} codes off"
        assert np.mean(lo != hi) < 1e-2  # the interval decides nearly every code
        norm = np.asarray(aux, dtype=np.float16).astype(np.float64).reshape(len(xr))
        n, rel = n[:, 0], rel[:, 0]
        assert np.all((norm >= ofmt.to_f16(n * (1 - rel))) & (norm <= ofmt.to_f16(n * (1 + rel))))
        return
    if fmt == "int4_g32":
        g = xr.reshape(len(xr), d // 32, 32)
        amax, t = np.max(np.abs(g), -1), tau
        s = np.asarray(aux, dtype=np.float16).astype(np.float64)
        one = 1 + 2.0 ** -22
        assert np.all((s >= ofmt.to_f16(np.maximum(amax - t, 0) / 7 / one)) & (s <= ofmt.to_f16((amax + t) / 7 * one)))
        q = ofmt.unpack_bits(rows, 4, d).reshape(g.shape).astype(np.int64) - 8
        s, t = s[..., None], tau[..., None] + 8 * 2.0 ** -23 * s[..., None]
        lo, hi = (np.clip(np.rint((g + sign * t) / s), -7, 7) for sign in (-1, 1))
        assert np.all((q >= lo) & (q <= hi))
        return
    if fmt == "fp16":
        rnd = lambda z: ofmt.to_f16(z).astype(np.float64)  # noqa: E731
        got = np.ascontiguousarray(rows).view(np.float16).astype(np.float64)
    else:
        rnd = lambda z: ofmt.e4m3_decode(ofmt.e4m3_encode(ofmt.to_f32(z)))  # noqa: E731
        got = ofmt.e4m3_decode(rows)
    assert np.all((got >= rnd(xr - tau)) & (got <= rnd(xr + tau)))


def run(fmt, d, t, hkv, rot, layout, ps=16, hq=4, kind="by_parts", scale=1.0, seed=0, q_shift=0):
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    kf, kb, vf, vb = fmt
    rng = np.random.default_rng([seed, d, t, rot])
    x = rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float32)
    x[:, hq:, rng.choice(d, 2, replace=False)] *= 30
    x = x.astype(np.float16)
    pos = rng.integers(0, 1 << 18, t).astype(np.int32)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    num_pages = (t + ps - 1) // ps + 3
    slots = rng.permutation(num_pages * ps)[:t].astype(np.int32)
    if t > 11:
        slots[7], slots[11] = -1, num_pages * ps + 5
    cache = kvq.PagedCache(d, hkv, num_pages, kf, vf, kb, vb, ks, vs, ps)
    canary = [(a, a.fill_(1)) for a in (cache.k_rows, cache.v_rows)]
    g = torch.from_numpy(x).cuda()
    q_buf, q_out = gu.guarded_empty(torch, (t, hq, d), torch.float16)
    kvq.kvq_rope_append(cache.struct, make_rope(kvq, rot, layout, kind, scale), torch.from_numpy(pos).cuda(),
                        g[:, hq:hq + hkv], g[:, hq + hkv:], torch.from_numpy(slots).cuda(), g[:, :hq], q_out)
    torch.cuda.synchronize()
    check_rope(q_out.cpu().numpy(), x[:, :hq], pos, rot, layout, kind, scale)
    gu.assert_guards(q_buf, q_out)
    keep = np.flatnonzero((slots >= 0) & (slots < num_pages * ps))
    untouched = np.setdiff1d(np.arange(num_pages * ps), slots[keep])
    for a, _ in canary:
        assert np.all(gu.pool_rows(a, untouched) == 1)
    turned = orope.apply(x[:, hq:hq + hkv], pos, frequencies(rot, kind), layout, scale)
    for side, (f, b, sg, rows, aux) in enumerate(((kf, kb, ks, cache.k_rows, cache.k_aux),
                                                  (vf, vb, vs, cache.v_rows, cache.v_aux))):
        rows = gu.pool_rows(rows, slots[keep])
        aux = None if aux is None else gu.pool_rows(aux, slots[keep])
        raw = x[keep, hq:hq + hkv] if side == 0 else x[keep, hq + hkv:]
        size = np.sum(np.abs(raw.astype(np.float64)), -1, keepdims=True)
        for h in range(hkv):
            xr = orot.rotate((turned[keep] if side == 0 else raw.astype(np.float64))[:, h], sg[h])
            tau = size[:, h] / math.sqrt(d) * (math.log2(d) + 2) * 2.0 ** -24
            if side == 0:
                tau = 2 * max(1.0, scale) * (tau + size[:, h] / math.sqrt(d) * 2.0 ** -21)
            check_side(xr, tau, f, b, rows[:, h], None if aux is None else aux[:, h])


# one warp per vector (a decode step), and the per-thread kernel (a chunk: over 16384 vectors)
@pytest.mark.parametrize("t,hkv", [(1, 1), (45, 3), (5600, 3), (2049, 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: f"{f[0]}{f[1] or ''}_{f[2]}{f[3] or ''}")
def test_formats(fmt, d, t, hkv):
    run(fmt, d, t, hkv, d, "half")


@pytest.mark.parametrize("t,hkv", [(45, 3), (5600, 3), (1400, 12)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 32), (64, 6), (128, 64), (128, 32), (128, 2), (128, 40), (128, 126), (256, 64),
                                   (256, 250), (256, 256)])
def test_rotated_parts(d, rot, layout, t, hkv):
    run(FORMATS[3], d, t, hkv, rot, layout, scale=1.2)


@pytest.mark.parametrize("t,hkv", [(45, 3), (5600, 3)])
@pytest.mark.parametrize("ps", [1, 12, 32])
def test_page_sizes(ps, t, hkv):
    run(FORMATS[0], 128, t, hkv, 128, "half", ps=ps)


@pytest.mark.parametrize("t", [33, 5700])
@pytest.mark.parametrize("fmt", ["codebook_qjl", "codebook_outlier"])
def test_sketched_and_outlier_keys(fmt, t):
    """Against the same call path with the keys turned first: kvq_quantize_append of the turned
    keys, of which the fused call differs only by not rounding them to fp16 (2^-11 relative):
    at most one code in fifty may differ, and norms by two fp16 ulps."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(t)
    hkv, d, ps = 3, 128, 16
    k = rng.standard_normal((t, hkv, d)).astype(np.float16)
    pos = torch.from_numpy(rng.integers(0, 1 << 16, t).astype(np.int32)).cuda()
    signs = np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8)
    proj = rng.standard_normal((128, d)).astype(np.float32) if fmt == "codebook_qjl" else None
    outl = np.stack([rng.choice(d, 8, replace=False) for _ in range(hkv)]).astype(np.int32)
    outl = outl if fmt == "codebook_outlier" else None
    pages = (t + ps - 1) // ps
    caches = [kvq.PagedCache(d, hkv, pages, fmt, "codebook", 3, 4, signs, signs, ps, k_qjl=proj, k_outliers=outl)
              for _ in range(2)]
    slots = torch.from_numpy(rng.permutation(pages * ps)[:t].astype(np.int32)).cuda()
    rope = make_rope(kvq, d, "half")
    kd = torch.from_numpy(k).cuda()
    kvq.kvq_rope_append(caches[0].struct, rope, pos, kd, kd, slots)
    turned = torch.empty_like(kd)
    kvq.kvq_rope_apply(rope, pos, kd, q_out=turned)
    caches[1].append(turned, kd, slots)
    torch.cuda.synchronize()
    a, b = (ofmt.unpack_bits(c.v_rows.cpu().numpy(), 4, d) for c in caches)
    assert np.mean(a != b) < gu.MAX_BOUNDARY_FRACTION and np.max(np.abs(a - b)) <= 1
    na, nb = (c.v_aux.cpu().numpy().view(np.uint16).astype(np.int64) for c in caches)
    assert np.max(np.abs(na - nb)) <= 1
    a, b = (ofmt.unpack_bits(gu.pool_rows(c.k_rows, np.arange(pages * ps))[..., :d * 3 // 8], 3, d) for c in caches)
    assert np.mean(a != b) < 0.02 and np.max(np.abs(a - b)) <= 1
    if fmt == "codebook_qjl":
        na, nb = (c.k_aux.cpu().numpy()[..., 0].view(np.uint16).astype(np.int64) for c in caches)
    else:
        na, nb = (ocache.unpack_outlier_aux(c.k_aux.cpu().numpy())[0].view(np.uint16).astype(np.int64) for c in caches)
    assert np.max(np.abs(na - nb)) <= 2


def test_sides_alone_queries_in_place_and_odd_query_rows():
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(2)
    t, hq, hkv, d = 9, 2, 2, 128
    signs = np.ones((hkv, d), dtype=np.int8)
    x = rng.standard_normal((t, hkv, d)).astype(np.float16)
    pos = rng.integers(0, 999, t).astype(np.int32)
    p, slots = torch.from_numpy(pos).cuda(), torch.arange(t, dtype=torch.int32, device="cuda")
    rope, xd = make_rope(kvq, d, "half"), torch.from_numpy(x).cuda()
    both, ks, vs = (kvq.PagedCache(d, hkv, 1, "codebook", "codebook", 4, 4, signs, signs) for _ in range(3))
    kvq.kvq_rope_append(both.struct, rope, p, xd, xd, slots)
    kvq.kvq_rope_append(ks.struct, rope, p, xd, None, slots)
    kvq.kvq_rope_append(vs.struct, rope, p, None, xd, slots)
    assert torch.equal(both.k_rows, ks.k_rows) and torch.equal(both.v_rows, vs.v_rows)
    assert not ks.v_rows.any() and not vs.k_rows.any()
    qx = rng.standard_normal((t, hq, d)).astype(np.float16)
    for shift in (0, 1):  # 16-byte rows in the same launch, others in one more
        flat = torch.zeros(qx.size + 8, dtype=torch.float16, device="cuda")
        q = flat[shift:shift + qx.size].view(qx.shape)
        q.copy_(torch.from_numpy(qx))
        kvq.kvq_rope_append(both.struct, rope, p, xd, xd, slots, q)
        check_rope(q.cpu().numpy(), qx, pos, d, "half")
    # a token without a slot still has its query turned
    q = torch.from_numpy(qx).cuda()
    kvq.kvq_rope_append(both.struct, rope, p, xd, xd, torch.full_like(slots, -1), q)
    check_rope(q.cpu().numpy(), qx, pos, d, "half")
    assert torch.equal(both.k_rows, ks.k_rows)


def test_capture_and_replay():
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(4)
    t, hkv, d = 12, 2, 128
    signs = np.ones((hkv, d), dtype=np.int8)
    x = torch.from_numpy(rng.standard_normal((t, hkv, d)).astype(np.float16)).cuda()
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    rope = make_rope(kvq, d, "half")
    eager, graphed = (kvq.PagedCache(d, hkv, 4, "fp8_e4m3", "int4_g32", 0, 0, signs, signs) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_rope_append(graphed.struct, rope, pos, x, x, slots)
    for step in range(3):  # positions and slots move on in place
        kvq.kvq_rope_append(eager.struct, rope, pos, x, x, slots)
        graph.replay()
        pos += 1
        slots += t
    torch.cuda.synchronize()
    assert torch.equal(eager.k_rows, graphed.k_rows) and torch.equal(eager.v_rows, graphed.v_rows)


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: f"{f[0]}{f[1] or ''}_{f[2]}{f[3] or ''}")
@pytest.mark.parametrize("d,t,hkv", [(64, 40, 3), (64, 5601, 3), (128, 40, 3), (128, 2049, 9), (256, 2050, 9)])
def test_values_that_are_not_finite_stay_in_their_vector(fmt, d, t, hkv):
    """Infinities and NaN in some vectors: every other vector's row is what it is without them, in
    both kinds of append (kvq_quantize_append too), and a codebook's norm tells which are bad."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    kf, kb, vf, vb = fmt
    rng = np.random.default_rng(d + t)
    x = rng.standard_normal((t, hkv, d)).astype(np.float16)
    bad = [(0, 0), (1, hkv - 1), (t // 2, 1), (t - 1, hkv - 1)]
    y = x.copy()
    for (i, h), v in zip(bad, (np.nan, np.inf, -np.inf, np.nan)):
        y[i, h, int(rng.integers(d))] = v
    y[t // 2, 1, :2] = np.inf, -np.inf
    pos = torch.from_numpy(rng.integers(0, 1 << 16, t).astype(np.int32)).cuda()
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    pages = (t + 15) // 16
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    rope = make_rope(kvq, d, "half")
    for fused in (True, False):
        got = []
        for z in (x, y):
            cache = kvq.PagedCache(d, hkv, pages, kf, vf, kb, vb, ks, vs)
            zd = torch.from_numpy(z).cuda()
            if fused:
                kvq.kvq_rope_append(cache.struct, rope, pos, zd, zd, slots)
            else:
                cache.append(zd, zd, slots)
            torch.cuda.synchronize()
            got.append([None if a is None else gu.pool_rows(a, np.arange(t))
                        for a in (cache.k_rows, cache.v_rows, cache.k_aux, cache.v_aux)])
        well = np.ones((t, hkv), bool)
        for i, h in bad:
            well[i, h] = False
        for side, (a, b) in enumerate(zip(*got)):
            if a is None:
                continue
            assert np.array_equal(a[well].view(np.uint8), b[well].view(np.uint8))
            if side >= 2 and (kf, vf)[side - 2] == "codebook":
                assert not np.isfinite(b[~well].astype(np.float32)).any()
