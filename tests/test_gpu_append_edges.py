"""What the two appends (kvq_quantize_append, kvq_rope_append; a warp per vector, and the per-thread
kernels above 16384 vectors) store for values at the ends of their formats."""
import numpy as np
import pytest

from oracle import cache as ocache
from tests import gpu_util as gu
from tests.test_gpu_rope import make_rope

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
