"""How far kvq_chunk_attention's outputs are off, as the header states it (2-norm over a call's outputs,
against the float64 oracle on the same bytes).

u = 2^-11.  A rounding to fp16 is off by u / sqrt(3) of a number at most in the mean square (0.43 u
over mantissas).  On vectors of independent normal coordinates, in squares: the output 0.43 u; weights
0.43 u, as their errors are independent and the output is their sum; values, or the centroids in
their place, 0.43 u; scores, sums of D products each off by 0.43 u (centroids) at variance 1, 0.43 u of
the weights again; of codebooks beside other tiers, a value's norm times its table's scale, 0.43 u.
Together sqrt(5) 0.43 u = 0.96 u: held to u.  Where some channels are thirty times the others, a key's norm is three times as
large or more and its scores with it; at three times, sqrt(4 + 9) 0.43 u = 1.55 u: held to that (keys that are
stored as they are multiplied have no such error, and the scale of a codebook's table is chosen for these)."""
import numpy as np
import pytest

from oracle import chunk as ochunk
from tests.test_gpu_chunk import Case, modules

pytestmark = pytest.mark.gpu
U = 2.0 ** -11
FORMATS = [(name, d) for name in ("fp16", "fp8_int4", "fp8_fp16", "cb4", "cb32", "cb23") for d in (64, 128, 256)]
FORMATS += [("qjl", 128), ("outlier", 128), ("outlier", 256), ("cb4+fp16", 128), ("cb32+fp8_int4", 256), ("cb4+fp16", 64)]


def relative_error(c, got):
    want = ochunk.chunk_attention(c.q, c.tiers, c.offsets, c.window, c.sinks)
    return float(np.linalg.norm(got.astype(np.float64) - want) / np.linalg.norm(want))


@pytest.mark.parametrize("name,d", FORMATS)
@pytest.mark.parametrize("group,count,lens", [(1, 9, 1500), (8, 70, 400), (2, 30, 40)])
@pytest.mark.parametrize("outliers", [False, True])
def test_error_of_the_outputs(name, d, group, count, lens, outliers):
    torch, kvq = modules()
    large = np.where(np.random.default_rng(d + count).random((2, 2, d)) < 0.01, 30.0, 1.0).astype(np.float16)

    def edit(tier, b, k, v):
        if outliers:
            k *= large[0]
            v *= large[1]
    if name in ("qjl", "outlier"):
        group = min(group, 4)  # (the codebook kernels, which such keys need, have no eight)
    specs = name.split("+")
    c = Case(kvq, torch, specs, [[lens]] if len(specs) == 1 else [[lens - 37], [37]], [count], hq=2 * group, hkv=2, d=d, seed=group,
             edit=edit)
    assert relative_error(c, c.run(kvq, torch)) <= (1.55 if outliers else 1.0) * U
