"""GPU parity of kvq_dequantize against the oracle's decoder, on bytes that the oracle wrote.

Tolerance, derived before the first run.  The kernel's rotated coordinates are exact stored
values times one float32 scale (2^-23 relative: the scale's own rounding and the product);
with a sketch, 128 float32 additions of S_j follow (128 2^-24 relative to the sum of their
sizes) and one fused multiply-add.  The transform adds (log2 D + 2) 2^-24 of sum|x~| / sqrt(D).
The result is rounded once to fp16: 2^-11 relative, or 2^-25 below the normal range."""
import math

import numpy as np
import pytest

import workloads as W
from oracle import cache as ocache
from oracle import formats as ofmt
from oracle import rotation as orot
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

SPECS = {
    "cb4": W.Tier("codebook", "codebook", 4, 4),
    "cb32": W.Tier("codebook", "codebook", 3, 2),
    "cb23u": W.Tier("codebook", "codebook", 2, 3, codebook="uniform"),
    "fp16": W.Tier("fp16", "fp16"),
    "fp8_int4": W.Tier("fp8_e4m3", "int4_g32"),
    "qjl": W.Tier("codebook_qjl", "codebook", 3, 4),
    "outlier": W.Tier("codebook_outlier", "codebook", 4, 4),
}


def build(kvq, torch, spec, n, hkv, d, ps, seed=0):
    rng = np.random.default_rng([seed, n, d])
    k, v = (rng.standard_normal((n, hkv, d)).astype(np.float32) for _ in range(2))
    k[:, :, rng.choice(d, 3, replace=False)] *= 30
    if n > 4:
        k[1], v[2] = 0.0, 0.0
        v[3] *= 1e-3
    k, v = k.astype(np.float16), v.astype(np.float16)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    proj = rng.standard_normal((ocache.QJL_DIM, d)).astype(np.float32)
    outl = ocache.outlier_channels(k) if spec.k_format == "codebook_outlier" else None
    b = gu.build_exact(kvq, torch, [spec], [[(k, v)]], ks, vs, ps, shuffle_seed=seed, k_qjl=proj, k_outl=outl)
    return b, proj


def expect(side, slots, h, ps, proj=None):
    """(value, error allowed before the fp16 rounding), float64 [T, d]."""
    page, off = slots // ps, slots % ps
    rows = side.rows[page, h, off]
    aux = None if side.aux is None else side.aux[page, h, off]
    d = side.signs.shape[-1]
    rot = ocache.decode_rotated(rows, aux, side.fmt, d, side.bits, side.centroids32)
    err = 2.0 ** -23 * np.abs(rot)
    if side.fmt == "codebook_qjl":
        z = 2.0 * ofmt.unpack_bits(rows[..., d * side.bits // 8:], 1, ocache.QJL_DIM) - 1.0
        c = aux[..., 1].astype(np.float64)[:, None] * math.sqrt(math.pi / 2) / ocache.QJL_DIM
        s64 = proj.astype(np.float64)
        rot = rot + c * (z @ s64)
        err = err + (ocache.QJL_DIM + 4) * 2.0 ** -24 * c * np.sum(np.abs(s64), 0) + 2.0 ** -24 * np.abs(rot)
    x = orot.unrotate(rot, side.signs[h])
    err = (np.sum(err, -1, keepdims=True) + (math.log2(d) + 2) * 2.0 ** -24 * np.sum(np.abs(rot), -1, keepdims=True)) / math.sqrt(d)
    err = np.broadcast_to(err, x.shape).copy()
    if side.fmt == "codebook_outlier":
        _, scale, q = ocache.unpack_outlier_aux(aux)
        add = q.astype(np.float64) * scale.astype(np.float64)[:, None]
        at = np.asarray(side.outliers[h], dtype=np.int64)
        x[:, at] += add
        err[:, at] += 2.0 ** -23 * np.abs(add)
    return x, err


def check(got, side, slots, ps, proj=None):
    for h in range(got.shape[1]):
        want, err = expect(side, slots, h, ps, proj)
        tol = err * (1 + 2.0 ** -9) + np.abs(want) * 2.0 ** -11 * (1 + 2.0 ** -9) + 2.0 ** -25
        off = np.abs(got[:, h].astype(np.float64) - want)
        assert np.all(off <= tol), f"head {h}: worst {np.max(off - tol)} at {np.argwhere(off > tol)[0]}"


@pytest.mark.parametrize("name", sorted(SPECS))
@pytest.mark.parametrize("d,n,ps", [(64, 1, 16), (64, 211, 12), (128, 203, 16), (128, 1, 1), (256, 97, 7), (128, 2500, 16)])
def test_matches_oracle(name, d, n, ps):
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    spec = SPECS[name]
    if d == 64 and name in ("qjl", "outlier"):
        pytest.skip("these keys take head_dim 128 and 256")
    hkv = 3
    b, proj = build(kvq, torch, spec, n, hkv, d, ps)
    tier = b.ora[0]
    rng = np.random.default_rng(n)
    all_slots = (np.repeat(tier.block_table[0], ps) * ps + np.tile(np.arange(ps), tier.block_table.shape[1]))[:n]
    slots = rng.permutation(all_slots).astype(np.int32)
    slots = np.concatenate([slots, slots[:2]])  # the same token twice
    t = len(slots)
    k_buf, k_out = gu.guarded_empty(torch, (t, hkv, d), torch.float16)
    v_buf, v_out = gu.guarded_empty(torch, (t, hkv, d), torch.float16)
    kvq.kvq_dequantize(b.gpu[0].struct, torch.from_numpy(slots).cuda(), k_out, v_out)
    torch.cuda.synchronize()
    check(k_out.cpu().numpy(), tier.k, slots, ps, proj)
    check(v_out.cpu().numpy(), tier.v, slots, ps)
    gu.assert_guards(k_buf, k_out)
    gu.assert_guards(v_buf, v_out)


def test_skipped_slots_and_one_side():
    """Slots outside the pool leave their rows as they were; either side alone."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    b, _ = build(kvq, torch, SPECS["cb4"], 40, 2, 128, 16)
    tier, c = b.ora[0], b.gpu[0]
    good = (tier.block_table[0][0] * 16 + np.arange(4)).astype(np.int32)
    slots = np.array([good[0], -1, good[1], c.num_pages * 16, good[2], 2 ** 31 - 1, -2 ** 31, good[3]], dtype=np.int32)
    live = np.array([0, 2, 4, 7])
    dead = np.array([1, 3, 5, 6])
    s = torch.from_numpy(slots).cuda()
    for side, kw in ((tier.k, "k_out"), (tier.v, "v_out")):
        out = torch.full((8, 2, 128), 7.5, dtype=torch.float16, device="cuda")
        kvq.kvq_dequantize(c.struct, s, **{kw: out})
        got = out.cpu().numpy()
        check(got[live], side, slots[live], 16)
        assert np.all(got[dead] == 7.5)


def test_write_then_read():
    """What kvq_quantize_append wrote comes back: fp16 rows within their rounding and the two
    rotations' float32 errors, the pair an identity up to (2 log2 D + 4) 2^-24 sum|x| / sqrt(D)
    a coordinate and the stored rounding, 2^-11 |x~| spread by the transform."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(3)
    t, hkv, d = 70, 2, 128
    signs = np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8)
    cache = kvq.PagedCache(d, hkv, 6, "fp16", "fp16", 0, 0, signs, signs)
    k, v = (rng.standard_normal((t, hkv, d)).astype(np.float16) for _ in range(2))
    slots = torch.from_numpy(rng.permutation(96)[:t].astype(np.int32)).cuda()
    cache.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots)
    ko, vo = (torch.empty((t, hkv, d), dtype=torch.float16, device="cuda") for _ in range(2))
    kvq.kvq_dequantize(cache.struct, slots, ko, vo)
    for got, x in ((ko, k), (vo, v)):
        x = x.astype(np.float64)
        rot = np.abs(orot.rotate(x, signs[None]))
        err = ((2 * math.log2(d) + 4) * 2.0 ** -24 * np.sum(np.abs(x), -1, keepdims=True)
               + np.sum(2.0 ** -11 * rot + 2.0 ** -25, -1, keepdims=True)) / math.sqrt(d)
        assert np.all(np.abs(got.cpu().numpy() - x) <= err * (1 + 2.0 ** -9) + 2.0 ** -11 * np.abs(x) * (1 + 2.0 ** -9) + 2.0 ** -25)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_int4_scales_near_the_largest(d):
    """Vectors along the signs put everything in one coordinate, 25000 sqrt(D): scales whose products
    with a level pass fp16's largest number, beside small ones."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(d)
    n, hkv, ps = 37, 3, 16
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    k, v = (rng.standard_normal((n, hkv, d)).astype(np.float16) for _ in range(2))
    for i in range(0, n, 3):
        v[i] = (25000.0 if i % 2 else 12000.0) * vs
    b = gu.build_exact(kvq, torch, [SPECS["fp8_int4"]], [[(k, v)]], ks, vs, ps, shuffle_seed=d)
    tier = b.ora[0]
    assert np.max(np.asarray(tier.v.aux).astype(np.float64)) > 8000
    t = np.arange(n)
    slots = (tier.block_table[0][t // ps] * ps + t % ps).astype(np.int32)
    out = torch.empty((n, hkv, d), dtype=torch.float16, device="cuda")
    kvq.kvq_dequantize(b.gpu[0].struct, torch.from_numpy(slots).cuda(), None, out)
    got = out.cpu().numpy()
    assert np.isfinite(got).all()
    check(got, tier.v, slots, ps)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("power", [-30, -7, 9, 30])
def test_codebooks_of_any_size(bits, power):
    """Centroids times a power of two, norms over it: the same vectors, to the bit."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(bits)
    t, hkv, d = 50, 2, 128
    signs = np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8)
    cache = kvq.PagedCache(d, hkv, 4, "codebook", "codebook", bits, bits, signs, signs)
    x = torch.from_numpy(rng.standard_normal((t, hkv, d)).astype(np.float16)).cuda()
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    cache.append(x, x, slots)
    want, got = torch.empty_like(x), torch.empty_like(x)
    kvq.kvq_dequantize(cache.struct, slots, want)
    if abs(power) < 10:  # norms are fp16: they take the factor back while they can
        cache.k_aux.mul_(2.0 ** -power)
        cache.k_centroids.mul_(2.0 ** power)
        kvq.kvq_dequantize(cache.struct, slots, got)
        assert torch.equal(got, want)
    else:  # the vectors leave fp16's range or its normal numbers
        cache.k_centroids.mul_(2.0 ** power)
        kvq.kvq_dequantize(cache.struct, slots, got)
        scaled = want.float() * 2.0 ** power
        if power > 0:
            big = scaled.abs() > 65520
            assert torch.isinf(got[big]).all()
        else:
            assert (got.float() - scaled).abs().max() <= 2.0 ** -24
