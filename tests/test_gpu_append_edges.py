"""What the two appends (kvq_quantize_append, kvq_rope_append; a warp per vector, and the per-thread
kernels above 16384 vectors) store for values at the ends of their formats."""
import numpy as np
import pytest

from oracle import cache as ocache
from oracle import formats as ofmt
from oracle import rope as orope
from tests import gpu_util as gu
from tests.test_gpu_rope import frequencies, make_rope

pytestmark = pytest.mark.gpu

SIZES = [(64, 40, 3), (64, 5601, 3), (128, 40, 3), (128, 2049, 9), (256, 40, 3), (256, 2050, 9)]


def store(kvq, torch, x, kf, vf, kb=0, vb=0, fused=True, scale=1.0, **kw):
    """x [T, Hkv, D] as keys (fused: turned by small positions) and as values; their pool rows."""
    t, hkv, d = x.shape
    rng = np.random.default_rng(hkv)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    cache = kvq.PagedCache(d, hkv, (t + 15) // 16, kf, vf, kb, vb, ks, vs, **kw)
    slots, xd = torch.arange(t, dtype=torch.int32, device="cuda"), torch.from_numpy(x).cuda()
    if fused:
        kvq.kvq_rope_append(cache.struct, make_rope(kvq, d, "half", scale=scale), slots % 100, xd, xd, slots)
    else:
        cache.append(xd, xd, slots)
    back = [torch.empty_like(xd) for _ in range(2)]
    kvq.kvq_dequantize(cache.struct, slots, *back)
    torch.cuda.synchronize()
    rows = [None if a is None else gu.pool_rows(a, np.arange(t)) for a in (cache.k_rows, cache.v_rows, cache.k_aux, cache.v_aux)]
    return rows, [b.cpu().numpy() for b in back]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("d,t,hkv", SIZES)
def test_a_nan_in_an_int4_vector_is_stored_as_nan(d, t, hkv, fused):
    """The rotation spreads it over the vector: every group's scale is NaN and every level 0, as the
    oracle has it, and the vector is read back as NaN.  Its neighbours are what they were."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(d + t)
    x = rng.standard_normal((t, hkv, d)).astype(np.float16)
    y = x.copy()
    bad = np.zeros((t, hkv), bool)
    for i, h in ((0, 0), (1, hkv - 1), (t // 2, 1), (t - 1, hkv - 1)):
        y[i, h, int(rng.integers(d))], bad[i, h] = np.nan, True
    _, oracle = ocache.encode(y[0, 0], np.ones(d), "int4_g32")
    assert np.isnan(oracle).all()
    want, back0 = store(kvq, torch, x, "int4_g32", "int4_g32", fused=fused)
    got, back = store(kvq, torch, y, "int4_g32", "int4_g32", fused=fused)
    for side in (0, 1):
        assert np.isnan(got[2 + side][bad]).all() and (got[side][bad] == 0x88).all()
        assert np.isnan(back[side][bad]).all()
        assert np.array_equal(got[side][~bad], want[side][~bad]) and np.array_equal(got[2 + side][~bad], want[2 + side][~bad])
        assert np.array_equal(back[side][~bad], back0[side][~bad])


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("t", [40, 5700])
def test_a_nan_in_an_outlier_channel_is_stored_as_nan(t, fused):
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(t)
    hkv, d = 3, 128
    outl = np.stack([rng.choice(d, 8, replace=False) for _ in range(hkv)]).astype(np.int32)
    x = rng.standard_normal((t, hkv, d)).astype(np.float16)
    x[t // 2, 1, outl[1, 3]] = np.nan
    rows, back = store(kvq, torch, x, "codebook_outlier", "codebook", 4, 4, fused, k_outliers=outl)
    _, scale, q = ocache.unpack_outlier_aux(rows[2])
    bad = np.zeros((t, hkv), bool)
    bad[t // 2, 1] = True
    assert np.isnan(scale[bad]).all() and not q[bad].any() and np.isfinite(scale[~bad]).all()
    assert np.isnan(back[0][t // 2, 1, outl[1]]).all() and np.isfinite(back[0][~bad]).all()


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 3), (256, 5)])
def test_a_codebook_vector_that_is_not_finite_has_codes_of_zero(d, hkv, bits):
    """NaN, infinities, and finite values whose sum of squares leaves float32: code 0 everywhere and a norm
    that is not finite, from both kernels of both appends."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(bits)
    for t in (40, 5700):
        for fused, scale in ((True, 1.0), (False, 1.0), (True, 1e30)):
            x = rng.standard_normal((t, hkv, d)).astype(np.float16)
            x[3, 1, 5], x[7, 2, d - 1], x[t - 1, 0, 0] = np.nan, np.inf, -np.inf
            x[20, 1, :2] = np.inf, -np.inf
            x[9, 0] = 0
            bad = ~np.isfinite(x).all(-1)
            rows, _ = store(kvq, torch, x, "codebook", "codebook", bits, bits, fused, scale=scale)
            for side in (0, 1):
                gone = bad if side or scale == 1.0 else x.any(-1)  # values are not scaled
                assert not rows[side][gone].any() and not np.isfinite(rows[2 + side][gone]).any()
                assert np.isfinite(rows[2 + side][~gone]).all() and rows[side][~gone].any(-1).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 36), (128, 128), (128, 50), (256, 256), (256, 100)])
def test_queries_in_place_in_the_same_launch(d, rot, layout):
    """Queries of a step turned in place, many heads to an SM, partners in other lanes: what they are out
    of place, to the bit, whatever lies beside them."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    t, hq, hkv = 150, 96, 2
    rng = np.random.default_rng(rot)
    signs = np.ones((hkv, d), dtype=np.int8)
    cache = kvq.PagedCache(d, hkv, 10, "fp16", "fp16", 0, 0, signs, signs)
    x = torch.from_numpy(rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float16)).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    rest = x[:, hq:].clone()
    pos = torch.from_numpy(rng.integers(0, 1 << 20, t).astype(np.int32)).cuda()
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    rope = make_rope(kvq, rot, layout)
    for _ in range(5):
        want = torch.empty(t, hq, d, dtype=torch.float16, device="cuda")
        kvq.kvq_rope_append(cache.struct, rope, pos, k, v, slots, q, want)
        kvq.kvq_rope_append(cache.struct, rope, pos, k, v, slots, q)
        assert torch.equal(q, want) and torch.equal(x[:, hq:], rest)


@pytest.mark.parametrize("quarters", [True, False])
@pytest.mark.parametrize("t", [1, 33, 5700])
@pytest.mark.parametrize("fmt", ["codebook_qjl", "codebook_outlier"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_side_data_of_turned_keys(fmt, t, layout, quarters):
    """Everything a key with a sketch or an outlier stream stores (codes, norm, sketch bits, residual norm;
    outlier scale and levels), against the oracle's encode of the turned key.

    Quarter turns: cos and sin are 0 and +-1, the turned key is an fp16 vector, and the criteria are
    those of kvq_quantize_append.  Any angle: a turned element is within (|a| + |b|) 2^-21 of the
    exact one.  That is far below a step of what is stored, so fp16 numbers differ by at most one
    step and levels by at most one; codes and sketch bits may differ where they are that close to a
    border: the error of u, about 2^-19, times the density of 7 borders and of the projections at theirs,
    below 1e-4 of them in either, and 1e-3 allowed.  Rows whose codes or norms differ have another
    residual (as in gu.check_qjl_rows): x~ - n C / sqrt(D) moves by a step of n, up to 2^-10 ||x~||,
    which is 2^-10 / 0.18 of a 3-bit residual's norm, six of its steps."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(t)
    hkv, d, ps, bits = 3, 128, 16, 3
    k = rng.standard_normal((t, hkv, d)).astype(np.float16)
    k[:, :, 11] *= 20
    pos = rng.integers(0, 1 << 16, t).astype(np.int32)
    signs = np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8)
    proj = rng.standard_normal((128, d)).astype(np.float32)
    outl = np.stack([rng.choice(d, 8, replace=False) for _ in range(hkv)]).astype(np.int32)
    pages = (t + ps - 1) // ps
    cache = kvq.PagedCache(d, hkv, pages, fmt, "codebook", bits, 4, signs, signs, ps, k_qjl=proj, k_outliers=outl)
    slots = rng.permutation(pages * ps)[:t].astype(np.int32)
    rope = make_rope(kvq, d, layout)
    if quarters:
        rope.turns.fill_(1 << 62)
    kd = torch.from_numpy(k).cuda()
    kvq.kvq_rope_append(cache.struct, rope, torch.from_numpy(pos).cuda(), kd, kd, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    rows, aux = gu.pool_rows(cache.k_rows, slots), gu.pool_rows(cache.k_aux, slots)
    if quarters:
        a, b = orope.pair_index(d, layout)
        turned = k.copy()
        c, s = (np.array(x)[pos % 4][:, None, None] for x in ([1, 0, -1, 0], [0, 1, 0, -1]))
        turned[..., a], turned[..., b] = k[..., a] * c - k[..., b] * s, k[..., b] * c + k[..., a] * s
        for h in range(hkv):
            if fmt == "codebook_qjl":
                gu.check_qjl_rows(turned[:, h], signs[h], bits, proj, rows[:, h], aux[:, h])
            else:
                gu.check_outlier_rows(turned[:, h], signs[h], bits, outl[h], rows[:, h], aux[:, h])
        return
    turned = orope.apply(k, pos, frequencies(d, "none"), layout)
    c32, b32 = gu.tables("lloyd_max", bits)
    step = lambda x, y: np.abs(x.view(np.int16).astype(int) - y.view(np.int16).astype(int))  # noqa: E731
    nb, off, all_bits = d * bits // 8, 0, 0
    for h in range(hkv):
        ro, ao = ocache.encode(turned[:, h], signs[h], fmt, bits, b32, c32, proj, outl[h])
        got = ofmt.unpack_bits(rows[:, h, :nb], bits, d) != ofmt.unpack_bits(ro[:, :nb], bits, d)
        assert np.mean(got) < 1e-3
        same = ~got.any(-1)
        if fmt == "codebook_qjl":
            assert step(aux[:, h, 0], ao[:, 0]).max() <= 1
            same &= aux[:, h, 0] == ao[:, 0]
            assert np.mean(same) > 0.9 or t == 1
            assert np.all(step(aux[same, h, 1], ao[same, 1]) <= 1)
            off += int(np.sum(ofmt.unpack_bits(rows[same, h, nb:], 1, 128) != ofmt.unpack_bits(ro[same, nb:], 1, 128)))
            all_bits += 128 * int(same.sum())
        else:
            for x, y in zip(ocache.unpack_outlier_aux(aux[:, h])[:2], ocache.unpack_outlier_aux(ao)[:2]):
                assert step(x, y).max() <= 1
            q, qo = (ocache.unpack_outlier_aux(z)[2].astype(int) for z in (aux[:, h], ao))
            assert np.abs(q - qo).max() <= 1 and np.mean(q != qo) < 0.02
    assert off <= 1e-3 * all_bits


@pytest.mark.parametrize("fmt,bits", [("codebook", 4), ("fp16", 0), ("int4_g32", 0)])
@pytest.mark.parametrize("d,t,hkv", SIZES)
def test_signs_at_other_addresses(d, t, hkv, fmt, bits):
    """Signs aligned to head_dim / 32 bytes only, whatever the size of the append: vectors within the
    float32 rounding of another kernel (codes and levels at a border)."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(d)
    x = torch.from_numpy(rng.standard_normal((t, hkv, d)).astype(np.float16)).cuda()
    signs = torch.from_numpy(np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8)).cuda()
    flat = torch.empty(hkv * d + 32, dtype=torch.int8, device="cuda")
    moved = flat[d // 32:d // 32 + hkv * d].view(hkv, d)
    moved.copy_(signs)
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    a, b = (kvq.PagedCache(d, hkv, (t + 15) // 16, fmt, fmt, bits, bits, s, s) for s in (signs, moved))
    for cache in (a, b):
        cache.append(x, x, slots)
    assert b.k_signs.data_ptr() % 16 == d // 32
    for m, n in ((a.k_rows, b.k_rows), (a.v_rows, b.v_rows)):
        assert (m != n).float().mean().item() < 1e-3
        if t == 40:
            assert torch.equal(m, n)
