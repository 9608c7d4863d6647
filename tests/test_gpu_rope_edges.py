"""Rotary positions where angles are small: slow pairs at the first positions of a sequence."""
import numpy as np
import pytest

from oracle import rope as orope
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("base", [1e4, 1e6, 1e8])
def test_small_angles_keep_their_sine(base, layout, transpose):
    """Pairs (0, b): the first element becomes -+ b sin(theta), with theta down to 1e-8.  Angle and sine are
    rounded to float32 (2^-24 and an ulp), the product once more and to fp16 (2^-11, 2^-25 where it is subnormal):
    2^-11 + 2^-21 of the value."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    d, hkv = 128, 2
    pos = np.array([0, 1, 2, 3, 5, 17, 100, -1, -2, -64], np.int32)
    rng = np.random.default_rng(int(base))
    x = np.zeros((len(pos), 3, d), np.float16)
    a, b = orope.pair_index(d, layout)
    x[..., b] = (rng.choice([-1, 1], (len(pos), 3, d // 2)) * rng.uniform(1000, 60000, (len(pos), 3, d // 2))).astype(np.float16)
    rope = kvq.Rope(d, layout, base)
    xd, p = torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda()
    out = torch.empty_like(xd)
    kvq.kvq_rope_apply(rope, p, xd, q_out=out, transpose=transpose)
    want = orope.apply(x, pos, orope.frequencies(base, d), layout, transpose=transpose)
    tol = np.abs(want) * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25
    assert np.all(np.abs(out.cpu().numpy() - want)[..., a] <= tol[..., a])
    if not transpose:  # queries of an append, the same angles
        signs = np.ones((hkv, d), dtype=np.int8)
        cache = kvq.PagedCache(d, hkv, 1, "fp16", "fp16", 0, 0, signs, signs)
        zero = torch.zeros(len(pos), hkv, d, dtype=torch.float16, device="cuda")
        slots = torch.arange(len(pos), dtype=torch.int32, device="cuda")
        kvq.kvq_rope_append(cache.struct, rope, p, zero, zero, slots, xd, out)
        assert np.all(np.abs(out.cpu().numpy() - want)[..., a] <= tol[..., a])
