"""GPU parity of kvq_rope_apply against the float64 oracle.

Tolerance, derived before the first run.  A coefficient (cos or sin times the scale s) carries:
the angle in half turns rounded to float32 (half a unit in the last place below 1: 2^-25,
times pi), its truncation to 32 bits (2 pi 2^-32), sincospi within one ulp (2^-24), the
scale's product (2^-25 s, scale at most 2 here): together below 2^-22 s.  The stored
frequency is within a few units of 2^-53 relative, times the angle (2^20 at most here):
2^-31.  A turned element is a product and a fused multiply-add, each rounded to 2^-24
relative: the float32 result is within (|a| + |b|) s (2^-22 + 2^-23) of the exact one, taken
as 2^-21, and is rounded once to fp16: half an ulp, 2^-11 relative, or 2^-25 below the normal
range."""
import numpy as np
import pytest

from oracle import rope as orope
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

SCALINGS = {"none": ("none", 1.0, 0.0, 0.0, 1.0), "linear": ("linear", 4.0, 0.0, 0.0, 1.0),
            "base": ("base", 8.0, 0.0, 0.0, 1.0), "by_parts": ("by_parts", 8.0, 8192.0, 1.0, 32.0)}


def frequencies(rot, kind):
    return orope.frequencies(10000.0, rot, *SCALINGS[kind])


def make_rope(kvq, rot, layout, kind="none", scale=1.0):
    k, factor, context, low, high = SCALINGS[kind]
    return kvq.Rope(rot, layout, 10000.0, k, factor, context, low, high, scale)


def check(got, x, pos, rot, layout, kind="none", scale=1.0, transpose=False):
    x = x.astype(np.float64)
    want = orope.apply(x, pos, frequencies(rot, kind), layout, scale, transpose)
    a, b = orope.pair_index(rot, layout)
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    tol = size * scale * 2.0 ** -21 + np.abs(want) * 2.0 ** -11 * (1 + 2.0 ** -9) + 2.0 ** -25
    tol[..., rot:] = 0.0  # copied
    off = np.abs(got.astype(np.float64) - want)
    assert np.all(off <= tol), f"{int(np.sum(off > tol))} elements off, worst {np.max(off - tol)}"


def inputs(t, hq, hkv, d, seed=0, far=1 << 20):
    rng = np.random.default_rng([seed, t, hq, d])
    x = rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float16)
    x[:, :, 3] *= 30
    pos = rng.integers(0, far, t).astype(np.int32)
    return x, pos


# (head_dim, rot): full, partial, sizes that no wide access fits, the smallest
ROTS = [(64, 64), (128, 128), (256, 256), (128, 64), (128, 32), (256, 128), (64, 16), (128, 2), (64, 6), (128, 48),
        (256, 250), (128, 40)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", ROTS)
@pytest.mark.parametrize("t", [1, 37])
def test_rope_views(t, d, rot, layout):
    """q and k as views of a fused projection, into dense outputs."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    hq, hkv = 6, 2
    x, pos = inputs(t, hq, hkv, d)
    rope = make_rope(kvq, rot, layout)
    g = torch.from_numpy(x).cuda()
    q_buf, q_out = gu.guarded_empty(torch, (t, hq, d), torch.float16)
    k_buf, k_out = gu.guarded_empty(torch, (t, hkv, d), torch.float16)
    kvq.kvq_rope_apply(rope, torch.from_numpy(pos).cuda(), g[:, :hq], g[:, hq:hq + hkv], q_out, k_out)
    torch.cuda.synchronize()
    check(q_out.cpu().numpy(), x[:, :hq], pos, rot, layout)
    check(k_out.cpu().numpy(), x[:, hq:hq + hkv], pos, rot, layout)
    gu.assert_guards(q_buf, q_out)
    gu.assert_guards(k_buf, k_out)
    assert np.array_equal(g.cpu().numpy(), x)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", sorted(SCALINGS))
@pytest.mark.parametrize("transpose", [False, True])
def test_scalings_and_transpose(kind, layout, transpose):
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    x, pos = inputs(53, 3, 1, 128, seed=2)
    rope = make_rope(kvq, 96, layout, kind, 1.25)
    out = torch.empty((53, 3, 128), dtype=torch.float16, device="cuda")
    kvq.kvq_rope_apply(rope, torch.from_numpy(pos).cuda(), torch.from_numpy(x).cuda()[:, :3], q_out=out,
                       transpose=transpose)
    check(out.cpu().numpy(), x[:, :3], pos, 96, layout, kind, 1.25, transpose)


@pytest.mark.parametrize("d,rot,shift", [(128, 128, 0), (128, 64, 0), (64, 64, 1), (128, 34, 0)])
def test_in_place_and_odd_addresses(d, rot, shift):
    """In place in a fused buffer, whose other heads stay; an address of two-byte alignment."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    t, hq, hkv = 29, 4, 2
    x, pos = inputs(t, hq, hkv, d, seed=3)
    flat = torch.zeros(x.size + 8, dtype=torch.float16, device="cuda")
    g = flat[shift:shift + x.size].view(x.shape)
    g.copy_(torch.from_numpy(x))
    kvq.kvq_rope_apply(make_rope(kvq, rot, "half"), torch.from_numpy(pos).cuda(), g[:, :hq], g[:, hq:hq + hkv])
    y = g.cpu().numpy()
    check(y[:, :hq + hkv], x[:, :hq + hkv], pos, rot, "half")
    assert np.array_equal(y[:, hq + hkv:], x[:, hq + hkv:])
    assert float(flat[:shift].abs().sum()) == 0 and float(flat[shift + x.size:].abs().sum()) == 0


def test_head_major_strides_and_many_tokens():
    """Inputs and outputs laid out [heads, tokens, d], more tokens than one block a token."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    t, h, d = 1500, 2, 64
    x, pos = inputs(t, h, 0, d, seed=4)
    g = torch.from_numpy(np.ascontiguousarray(x.transpose(1, 0, 2))).cuda().transpose(0, 1)
    out = torch.empty((h, t, d), dtype=torch.float16, device="cuda").transpose(0, 1)
    kvq.kvq_rope_apply(make_rope(kvq, d, "interleaved"), torch.from_numpy(pos).cuda(), g, q_out=out)
    check(out.cpu().numpy(), x, pos, d, "interleaved")


def test_far_and_negative_positions():
    """Exact reduction: at positions up to the largest int the angle is that of integer
    arithmetic on the stored fraction, and a negative position turns backwards."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    d = 128
    rope = make_rope(kvq, d, "half")
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321], dtype=np.int32)
    x = np.random.default_rng(9).standard_normal((len(pos), 1, d)).astype(np.float16)
    out = torch.empty((len(pos), 1, d), dtype=torch.float16, device="cuda")
    kvq.kvq_rope_apply(rope, torch.from_numpy(pos).cuda(), torch.from_numpy(x).cuda(), q_out=out)
    turns = [int(v) for v in kvq.kvq_rope_table(10000.0, d)]
    frac = np.array([[((int(p) * f) % 2 ** 64) / 2.0 ** 64 for f in turns] for p in pos])
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    a, b = x[..., :64].astype(np.float64), x[..., 64:].astype(np.float64)
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    tol = np.tile((np.abs(a) + np.abs(b)) * 2.0 ** -21, 2) + np.abs(want) * 2.0 ** -11 * (1 + 2.0 ** -9) + 2.0 ** -25
    assert np.all(np.abs(out.cpu().numpy() - want) <= tol)
    assert np.array_equal(out[0].cpu().numpy(), x[0])  # position 0 turns nothing


def test_gradient_against_differences():
    """The transpose is the gradient: <R(x + e) - R(x - e), g> / 2 = <e, R^T g> for a linear map,
    up to the fp16 rounding of each side's outputs (half an ulp of every element summed)."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    rng = np.random.default_rng(11)
    t, h, d = 5, 2, 128
    pos = torch.from_numpy(rng.integers(0, 5000, t).astype(np.int32)).cuda()
    rope = make_rope(kvq, d, "interleaved", "by_parts", 1.1)
    x, e, g = (torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float16)).cuda() for _ in range(3))

    def turn(v, transpose=False):
        out = torch.empty_like(v)
        kvq.kvq_rope_apply(rope, pos, v, q_out=out, transpose=transpose)
        return out.double()

    plus, minus = (x + e), (x - e)
    up, down, back = turn(plus), turn(minus), turn(g, True)
    exact_e = (plus.double() - minus.double()) / 2  # what the rounded inputs differ by
    lhs = ((up - down) / 2 * g.double()).sum()
    rhs = (exact_e * back).sum()
    half = 2.0 ** -11 * (1 + 2.0 ** -8)  # and the float32 terms
    room = (half * (up.abs() + down.abs()) / 2 * g.double().abs()).sum() + (half * back.abs() * exact_e.abs()).sum()
    assert abs(float(lhs - rhs)) <= float(room)


def test_capture_replay_and_streams():
    """Two captured graphs and eager calls on another stream, interleaved."""
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    x, pos = inputs(17, 4, 0, 128, seed=6)
    rope = make_rope(kvq, 128, "half")
    q = torch.from_numpy(x).cuda()
    p = torch.from_numpy(pos).cuda()
    outs = [torch.zeros_like(q) for _ in range(3)]
    graphs = []
    for o in outs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kvq.kvq_rope_apply(rope, p, q, q_out=o)
        graphs.append(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for graph in graphs:
        graph.replay()
    with torch.cuda.stream(side):
        kvq.kvq_rope_apply(rope, p, q, q_out=outs[2])
    torch.cuda.synchronize()
    for o in outs:
        check(o.cpu().numpy(), x, pos, 128, "half")
    q.copy_(torch.from_numpy(x * np.float16(0.5)))  # new inputs in the same place
    for graph in graphs:
        graph.replay()
    check(outs[0].cpu().numpy(), (x * np.float16(0.5)), pos, 128, "half")
