"""GPU parity of kvq_chunk_attention and kvq_decode_attention_window against the float64 oracle, on
bytes that the oracle wrote.

Tolerance, derived before the first run, u = 2^-11 (half a step of fp16, relative).  A score: queries
are two fp16 numbers (2^-22), a decoded key is rounded at most three times (table entry; the sum with a sketch's
estimate or an outlier stream; an INT4 value once), so with S_t = sum_i |q~_i| |k~_ti| / sqrt(D) it is off
by at most 3 u S_t (1 + 2^-9), and float32 accumulation of 2 D products stays below 2^-15 S_t.  A weight is off by
the factor e^d, d = the largest of that, twice (numerator and denominator), and is rounded to fp16 (u, or
2^-25 absolute below 2^-14 where the running maximum's weight is at least 2^-8 and at most 4: 2^-25 2^8 of
the largest weight, times its number of tokens at most).  The values are rounded at most twice (2 u of
|v~|_2 a coordinate, the inverse rotation being orthogonal), the output once.  The bound is the
worst case; independent roundings add in squares, so the 2-norm over all outputs is held to 2^-9 of
the outputs' besides (scores u sqrt(3), weights u, values u sqrt(2), output u: under 3 u, 4 u allowed)."""
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import cache as ocache
from oracle import chunk as ochunk
from oracle import rotation as orot
from tests import gpu_util as gu
from tests.test_gpu_shared import SPECS

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


def modules():
    return gu.torch_cuda(), gu.kvq_module()


def estimate(tier, b, g, n):
    """The sketch's estimate of the residuals of n tokens, rotated [n, d] (zeros without a sketch)."""
    d = tier.k.signs.shape[1]
    if tier.k.fmt != ocache.CODEBOOK_QJL or n == 0:
        return np.zeros((n, d))
    rows, aux = ocache.gather(tier.k, tier.block_table[b], n, g, tier.page_size)
    return np.stack([ocache.qjl_correction(rows, aux, e, tier.k.proj, d, tier.k.bits) for e in np.eye(d)], -1)


class Case:
    def __init__(self, kvq, torch, specs, lens, counts, hq, hkv, d=128, ps=16, window=0, sinks=0, seed=0, spread=1.0,
                 edit=None):
        """specs: tier names, oldest first; lens: per tier, a length per sequence; counts: new tokens of
        each sequence; edit(tier, sequence, k, v) may change the vectors before they are stored."""
        rng = np.random.default_rng([seed, hq, hkv, d, ps])
        kv = []
        for t, per in enumerate(lens):
            kv.append([])
            for b, n in enumerate(per):
                k, v = ((rng.standard_normal((n, hkv, d)) * x).astype(np.float16) for x in (spread, 1.0))
                if edit:
                    edit(t, b, k, v)
                kv[-1].append((k, v))
        ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
        proj = rng.standard_normal((128, d)).astype(np.float32)
        outl = np.stack([rng.choice(d, 8, replace=False) for _ in range(hkv)]).astype(np.int32)
        self.built = gu.build_exact(kvq, torch, [SPECS[s] for s in specs], kv, ks, vs, ps, shuffle_seed=seed + 1,
                                    k_qjl=proj, k_outl=outl)
        first = self.built.gpu[0].struct
        for c in self.built.gpu[1:]:  # one set of signs and one projection, as the calls want it
            c.struct.k_signs, c.struct.v_signs = first.k_signs, first.v_signs
            if c.struct.k_qjl and first.k_qjl:
                c.struct.k_qjl = first.k_qjl
        self.views, self.tiers = self.built.views, self.built.ora
        self.offsets = [0] + [int(x) for x in np.cumsum(counts)]
        self.batch, self.hq, self.hkv, self.d, self.window, self.sinks = len(counts), hq, hkv, d, window, sinks
        self.q = rng.standard_normal((self.offsets[-1], hq, d)).astype(np.float16)

    def run(self, kvq, torch, q=None, out=None, decode=False, offsets=None, bits=0, fill=0xFF):
        q = torch.from_numpy(self.q).cuda() if q is None else q
        n = q.shape[0]
        need = (kvq.kvq_decode_window_workspace_size(self.views, self.batch, self.hq, self.window, self.sinks) if decode
                else kvq.kvq_chunk_workspace_size(self.views, self.batch, n, self.hq, self.window, self.sinks))
        out_buf = None
        if out is None:
            out_buf, out = gu.guarded_empty(torch, tuple(q.shape), torch.float16)
            out.fill_(7.0)
        ws_buf, ws = gu.guarded_empty(torch, (need,), torch.uint8)
        ws.fill_(fill)  # what a workspace holds does not matter
        status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        if decode:
            kvq.kvq_decode_attention_window(self.views, q, out, ws, self.window, self.sinks, status=status)
        else:
            off = torch.tensor(self.offsets if offsets is None else offsets, dtype=torch.int32, device="cuda")
            kvq.kvq_chunk_attention(self.views, off, q, out, ws, self.window, self.sinks, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == bits, f"device error bits {int(status.item())}"
        if out_buf is not None:
            gu.assert_guards(out_buf, out)
        gu.assert_guards(ws_buf, ws)
        return out.cpu().numpy()

    def check(self, got, tokens=None, offsets=None):
        """tokens: of q, the ones to look at (all by default)."""
        grp, sum_off, sum_size = self.hq // self.hkv, 0.0, 0.0
        offsets = self.offsets if offsets is None else offsets
        for b in range(self.batch):
            count, length = offsets[b + 1] - offsets[b], sum(int(t.lens[b]) for t in self.tiers)
            todo = [i for i in range(count) if tokens is None or offsets[b] + i in tokens]
            for g in range(self.hkv) if todo else ():
                keys, values = oatt.dequantised_kv(self.tiers, b, g)
                if keys is None:
                    assert not got[offsets[b]:offsets[b + 1], g * grp:(g + 1) * grp].any()
                    continue
                signs = self.built.k_signs[g]
                k = np.abs(orot.rotate(keys, signs) + np.concatenate([estimate(t, b, g, int(t.lens[b])) for t in self.tiers]))
                size = np.linalg.norm(values, axis=-1)
                for i in todo:
                    seen = ochunk.sees(length - count + i, length, self.window, self.sinks)
                    for h in range(g * grp, (g + 1) * grp):
                        y = got[offsets[b] + i, h].astype(np.float64)
                        if not seen.any():
                            assert not y.any()
                            continue
                        q = self.q[offsets[b] + i, h].astype(np.float64)
                        s = ((keys @ q + oatt.sketch_terms(self.tiers, b, g, q)) / math.sqrt(self.d))[seen]
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        v = values[seen]
                        want = w @ v
                        off = float(np.max((3 * U * (1 + 2.0 ** -9) + 2.0 ** -15) * (k[seen] @ np.abs(orot.rotate(q, signs))))) / math.sqrt(self.d)
                        tol = (2 * math.expm1(off) + U) * (w @ np.abs(v)) + 2 * U * (w @ size[seen])
                        tol = (tol + 2.0 ** -17 * w.max() * len(w) * np.max(np.abs(v))) * (1 + 2.0 ** -9) + U * np.abs(want) + 2.0 ** -25
                        bad = ~(np.abs(y - want) <= tol)
                        assert not bad.any(), f"token {i} of {b}, head {h}: {int(bad.sum())} off, worst {np.max(np.abs(y - want) / tol)}"
                        sum_off += float(np.sum((y - want) ** 2))
                        sum_size += float(np.sum(want ** 2))
        rel = math.sqrt(sum_off / max(sum_size, 1e-300))
        assert sum_size == 0 or rel <= 2.0 ** -9, f"relative error {rel}"


@pytest.mark.parametrize("context,count", [(0, 1), (0, 2), (1, 1), (15, 1), (16, 3), (127, 2), (100, 29), (128, 128), (255, 130),
                                           (1000, 5), (0, 300), (513, 64)])
def test_lengths(context, count):
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16"], [[context + count]], [count], hq=4, hkv=2, seed=context + count)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "fp8_fp16", "cb4", "cb32", "cb23"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_formats_and_groups(name, group):
    """With the second sequence unpacked, where it has the rows."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[400, 140, 33]], [17, 70, 33], hq=2 * group, hkv=2, seed=group)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name", ["fp8_int4", "cb4"])
@pytest.mark.parametrize("count", [511, 512, 513, 700])
def test_where_unpacking_begins(name, count):
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[900, 800, 20]], [count, 8, 20], hq=2, hkv=2, seed=count)
    c.check(c.run(kvq, torch), set(range(0, count, 37)) | set(range(count - 3, count + 28)))


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "fp8_fp16", "cb4", "cb32", "cb23"])
@pytest.mark.parametrize("d", [64, 256])
def test_head_dims(name, d):
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[333, 70, 200]], [40, 70, 1], hq=4, hkv=2, d=d, seed=d)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name,d,group", [("qjl", 128, 2), ("outlier", 128, 4), ("outlier", 256, 1)])
def test_keys_with_extra(name, d, group):
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[200, 31]], [9, 5], hq=2 * group, hkv=2, d=d, seed=3)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name,d,hq", [("fp16", 128, 2), ("cb4", 128, 2), ("fp16", 128, 4), ("cb4", 128, 4), ("fp8_int4", 64, 2),
                                       ("cb32", 256, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 128), (129, 3), (300, 200), (5000, 10)])
def test_windows(name, d, hq, window, sinks):
    """Windows and sinks that begin and end inside pages and tiles, meet one another, or hold everything."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[700, 90]], [150, 20], hq=hq, hkv=1, d=d, window=window, sinks=sinks, seed=window)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name,d", [("fp16", 128), ("fp8_int4", 128), ("cb4", 128), ("cb32", 128), ("cb4", 256), ("fp16", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 4), (1000, 1)])
def test_decode_window(name, d, window, sinks):
    """The decode form, and the chunk call with one token a sequence."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[700, 0, 1, 65, 300]], [1] * 5, hq=8, hkv=2, d=d, window=window, sinks=sinks, seed=window)
    got = c.run(kvq, torch, decode=True)
    c.check(got)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name,d,group", [("qjl", 128, 1), ("qjl", 128, 4), ("outlier", 128, 4), ("outlier", 256, 1),
                                          ("cb4", 128, 1), ("cb23", 128, 2), ("cb4", 128, 8), ("cb32", 256, 8), ("cb32", 256, 1),
                                          ("fp16", 128, 1), ("fp16", 128, 8), ("fp8_int4", 128, 8), ("fp8_fp16", 128, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 5)])
def test_decode_window_of_every_kernel(name, d, group, window, sinks):
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[200, 31, 38, 0, 39]], [1] * 5, hq=2 * group, hkv=2, d=d, window=window, sinks=sinks, seed=group)
    c.check(c.run(kvq, torch, decode=True))


@pytest.mark.parametrize("ps", [1, 3, 24, 128, 200])
@pytest.mark.parametrize("name", ["fp8_int4", "cb32"])
def test_decode_window_page_sizes(name, ps):
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[301, 50, 155]], [1] * 3, hq=4, hkv=2, ps=ps, window=100, sinks=7, seed=ps)
    c.check(c.run(kvq, torch, decode=True))


@pytest.mark.parametrize("specs,lens", [(["fp8_int4", "fp16"], [[300, 0, 128, 7], [64, 33, 0, 1]]),
                                        (["cb4", "fp16"], [[300, 0, 128, 7], [64, 33, 0, 1]]),
                                        (["cb32", "cb4", "fp8_int4", "fp16"], [[130, 5, 0, 16], [100, 0, 2, 16], [40, 7, 0, 16], [50, 1, 1, 16]])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 9), (5, 200), (30, 140)])
@pytest.mark.parametrize("hq", [4, 16])
def test_tiers(specs, lens, window, sinks, hq):
    """Tokens of several tiers, one tier after the other; chunks that reach across them, and tiers that a sequence has not."""
    torch, kvq = modules()
    counts = [80, 20, 2, 3]
    c = Case(kvq, torch, specs, lens, counts, hq=hq, hkv=2, window=window, sinks=sinks, seed=len(specs))
    c.check(c.run(kvq, torch))
    c = Case(kvq, torch, specs, lens, [1] * 4, hq=hq, hkv=2, window=window, sinks=sinks, seed=len(specs))
    c.check(c.run(kvq, torch))
    c.check(c.run(kvq, torch, decode=True))


@pytest.mark.parametrize("ps", [1, 3, 8, 24, 128, 200])
def test_page_sizes(ps):
    torch, kvq = modules()
    for name in ("fp8_int4", "cb32"):
        c = Case(kvq, torch, [name], [[301, 50]], [33, 2], hq=4, hkv=2, ps=ps, window=150, sinks=5, seed=ps)
        c.check(c.run(kvq, torch))


def test_ragged_batch():
    """Sequences without new tokens, without any token, and chunks longer than what is cached."""
    torch, kvq = modules()
    lens, counts = [0, 5, 300, 140, 1, 0, 129, 77], [3, 0, 20, 140, 1, 0, 300, 80]
    for name in ("fp16", "cb4"):
        c = Case(kvq, torch, [name], [lens], counts, hq=8, hkv=2, seed=5)
        c.check(c.run(kvq, torch))


@pytest.mark.parametrize("batch", [40, 1500])
def test_many_sequences(batch):
    """More sequences than one pass of the plan takes; a few are looked at."""
    torch, kvq = modules()
    rng = np.random.default_rng(batch)
    lens, counts = rng.integers(0, 40, batch), rng.integers(0, 4, batch)
    c = Case(kvq, torch, ["fp16"], [lens], counts, hq=2, hkv=1, d=64, ps=16, seed=batch)
    look = set(range(0, c.offsets[-1], max(1, c.offsets[-1] // 97))) | {c.offsets[-1] - 1}
    c.check(c.run(kvq, torch), look)


def test_strided_heads_and_in_place():
    """Queries out of a fused projection's output, outputs in another's, heads before tokens, and in place."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[200, 90]], [30, 7], hq=4, hkv=2, seed=9)
    n, q = c.offsets[-1], torch.from_numpy(c.q).cuda()
    plain = c.run(kvq, torch)
    c.check(plain)
    qkv = torch.randn((n, 8, 128), device="cuda").half()
    qkv[:, 2:6] = q
    wide = torch.full((n, 9, 136), 3.0, dtype=torch.float16, device="cuda")
    got = c.run(kvq, torch, q=qkv[:, 2:6], out=wide[:, 1:5, 8:])
    assert np.array_equal(got, plain)
    wide[:, 1:5, 8:] = 3.0
    assert bool((wide == 3.0).all())  # nothing beside the heads was written
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert np.array_equal(c.run(kvq, torch, q=turned, out=torch.empty((4, n, 128), dtype=torch.float16, device="cuda").transpose(0, 1)), plain)
    keep = qkv.clone()
    assert np.array_equal(c.run(kvq, torch, q=qkv[:, 2:6], out=qkv[:, 2:6]), plain)
    assert torch.equal(qkv[:, :2], keep[:, :2]) and torch.equal(qkv[:, 6:], keep[:, 6:])


def test_padded_tokens_are_left_alone():
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb4"], [[50, 60, 9]], [4, 6, 2], hq=4, hkv=2, seed=2)
    q = torch.cat([torch.from_numpy(c.q).cuda(), torch.full((20, 4, 128), float("nan"), dtype=torch.float16, device="cuda")])
    got = c.run(kvq, torch, q=q)
    c.check(got[:12])
    assert (got[12:] == 7.0).all()
    # and before the first chunk
    shifted = [x + 3 for x in c.offsets]
    q = torch.cat([q[:3] * 0, torch.from_numpy(c.q).cuda()])
    got = c.run(kvq, torch, q=q, offsets=shifted)
    c.check(got[3:])
    assert (got[:3] == 7.0).all()


def test_offsets_out_of_order_are_reported():
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16"], [[50, 60, 40]], [4, 6, 2], hq=4, hkv=2, seed=2)
    for off, used in [([0, 4, 3, 12], [0, 4, 4, 12]), ([-2, 4, 10, 12], [0, 4, 10, 12]), ([0, 4, 10, 99], [0, 4, 10, 12]),
                      ([0, 50, 10, 12], [0, 12, 12, 12])]:
        got = c.run(kvq, torch, offsets=off, bits=kvq.DEVERR_OFFSETS)
        c.check(got, offsets=used)


def test_lengths_and_pages_out_of_range_are_reported():
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16"], [[50, 60]], [4, 6], hq=4, hkv=2, seed=2)
    want = c.run(kvq, torch)
    c.views[0].seq_lens[0] = 1 << 20
    got = c.run(kvq, torch, bits=kvq.DEVERR_SEQ_LEN)
    assert np.array_equal(got[4:], want[4:]) and np.isfinite(got[:4].astype(np.float64)).all()
    c.views[0].seq_lens[0] = -5
    got = c.run(kvq, torch, bits=kvq.DEVERR_SEQ_LEN)
    assert np.array_equal(got[4:], want[4:]) and not got[:4].any()
    c.views[0].seq_lens[0] = 50
    for bad in (-1, 1 << 30, c.built.gpu[0].num_pages):
        page = int(c.views[0].block_table[0, 1])
        c.views[0].block_table[0, 1] = bad
        got = c.run(kvq, torch, bits=kvq.DEVERR_PAGE_INDEX)
        assert np.array_equal(got[4:], want[4:])
        c.views[0].block_table[0, 1] = page
    assert np.array_equal(c.run(kvq, torch), want)


def nan_at(positions, side):
    def edit(tier, b, k, v):
        for t, value in positions:
            (k if side == "k" else v)[t, :, 3] = value
    return edit


@pytest.mark.parametrize("name,d,group", [("fp16", 128, 2), ("cb4", 128, 2), ("fp8_int4", 128, 2), ("fp8_fp16", 128, 1),
                                          ("fp16", 128, 8), ("cb4", 128, 8), ("fp8_int4", 128, 8), ("fp16", 64, 2), ("cb32", 256, 2)])
@pytest.mark.parametrize("side", ["k", "v"])
def test_what_a_query_does_not_see_does_not_reach_it(name, d, group, side):
    """Vectors that are not finite, behind a query, before its window, and (in pages) behind the sequence; on
    packed tiles and (eight heads a kv head; other head_dims) on unpacked ones."""
    torch, kvq = modules()
    bad = [(20, np.nan), (250, np.inf)]  # before the window of all queries; in the middle of the chunk
    args = dict(specs=[name], lens=[[300]], counts=[120], hq=group, hkv=1, d=d, window=130, sinks=4, seed=1)
    with np.errstate(invalid="ignore"):
        c = Case(kvq, torch, edit=nan_at([(t, 1.0) for t, _ in bad], side), **args)
        e = Case(kvq, torch, edit=nan_at(bad, side), **args)
    for cache in (c.built.gpu[0], e.built.gpu[0]):  # slots of no token
        held = torch.zeros(cache.num_pages, 16, dtype=torch.bool, device="cuda")
        t = torch.arange(300, device="cuda")
        held[c.views[0].block_table[0].long()[t // 16], t % 16] = True
        free = ~held[:, None, :].expand(-1, 1, -1)
        for rows in (cache.k_rows, cache.v_rows):
            rows[free] = 0x7E
        for aux in (cache.k_aux, cache.v_aux):
            if aux is not None:
                aux[free] = float("nan")
    want, got = c.run(kvq, torch), e.run(kvq, torch)
    c.check(want)
    # query i stands at 180 + i: it sees position 20 never (20 <= 180 - 130), position 250 from i = 70 on.  (The
    # others' results may differ in their last bit: running maxima are raised by the warp.)
    c.check(got[:70], set(range(70)))
    if side == "v":
        assert not np.isfinite(got[70:].astype(np.float64)).all(-1).any()


@pytest.mark.parametrize("name,d,group", [("fp16", 128, 4), ("fp16", 128, 8), ("fp8_int4", 128, 1), ("fp8_int4", 128, 4), ("fp8_fp16", 128, 2),
                                          ("cb4", 128, 1), ("cb4", 128, 4), ("cb4", 128, 8), ("cb32", 256, 1), ("cb32", 256, 2),
                                          ("qjl", 128, 1), ("qjl", 128, 2), ("outlier", 128, 2), ("outlier", 256, 1), ("fp16", 64, 2),
                                          ("cb4", 64, 2)])
@pytest.mark.parametrize("side", ["k", "v"])
def test_what_a_decode_window_hides_does_not_reach_it(name, d, group, side):
    """Vectors that are not finite on the pages where the sinks end and the window begins."""
    torch, kvq = modules()
    bad = [(4, np.nan), (15, np.inf), (160, np.nan), (169, -np.inf)]  # of 300 tokens the first 4 and the last 130 are seen
    args = dict(specs=[name], lens=[[300]], counts=[1], hq=group, hkv=1, d=d, window=130, sinks=4, seed=1)
    with np.errstate(invalid="ignore"):
        c = Case(kvq, torch, edit=nan_at([(t, 1.0) for t, _ in bad], side), **args)
        e = Case(kvq, torch, edit=nan_at(bad, side), **args)
    c.check(c.run(kvq, torch, decode=True))
    c.check(e.run(kvq, torch, decode=True))


@pytest.mark.parametrize("hq", [4, 16])
def test_a_query_that_is_not_finite_stays_alone(hq):
    torch, kvq = modules()
    for name in ("fp16", "cb4"):
        c = Case(kvq, torch, [name], [[200]], [70], hq=hq, hkv=2, seed=4)
        want = c.run(kvq, torch)
        q = torch.from_numpy(c.q).cuda()
        q[7, 1, 5], q[20, 3, 0] = float("nan"), float("inf")
        got = c.run(kvq, torch, q=q)
        assert np.isnan(got[7, 1].astype(np.float64)).all() and np.isnan(got[20, 3].astype(np.float64)).all()
        got[7, 1], got[20, 3] = want[7, 1], want[20, 3]
        c.check(got)


@pytest.mark.parametrize("name", ["fp16", "cb4", "fp8_int4"])
@pytest.mark.parametrize("count", [200, 400])  # (two query heads a kv head: packed and unpacked)
def test_large_scores_and_growing_maxima(name, count):
    """Scores that grow along the context, so that running maxima are raised again and again, and one token that outweighs all."""
    torch, kvq = modules()

    def edit(tier, b, k, v):
        k *= np.linspace(0.1, 4.0, len(k))[:, None, None].astype(np.float16)
        k[len(k) // 2] *= 6.0
    c = Case(kvq, torch, [name], [[900]], [count], hq=2, hkv=1, seed=6, edit=edit)
    c.check(c.run(kvq, torch), set(range(0, count, 7)))


def test_split_over_a_long_context():
    """Few queries on many tokens: the context is split; sampled queries."""
    torch, kvq = modules()
    for name in ("fp8_int4", "cb4"):
        c = Case(kvq, torch, [name], [[9000, 3000]], [3, 2], hq=2, hkv=1, seed=8)
        c.check(c.run(kvq, torch))


def test_twice_the_same():
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb32"], [[2000, 300]], [200, 20], hq=4, hkv=2, seed=8)
    assert np.array_equal(c.run(kvq, torch), c.run(kvq, torch, fill=0))


def test_captured_and_replayed_on_other_lengths():
    """A captured call reads lengths, offsets and block tables when it runs; two graphs share a workspace."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[400, 300]], [40, 30], hq=4, hkv=2, window=128, sinks=2, seed=3)
    q = torch.from_numpy(c.q).cuda()
    out, off = torch.zeros_like(q), torch.tensor(c.offsets, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(kvq.kvq_chunk_workspace_size(c.views, 2, 70, 4, 128, 2),
                         kvq.kvq_decode_window_workspace_size(c.views, 2, 4, 128, 2)), dtype=torch.uint8, device="cuda")
    one = torch.zeros((2, 4, 128), dtype=torch.float16, device="cuda")

    def both():
        kvq.kvq_chunk_attention(c.views, off, q, out, ws, 128, 2)
        kvq.kvq_decode_attention_window(c.views, last, one, ws, 128, 2)
    last = q[[39, 69]].contiguous()
    both()
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: kvq.kvq_chunk_attention(c.views, off, q, out, ws, 128, 2),
                 lambda: kvq.kvq_decode_attention_window(c.views, last, one, ws, 128, 2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for offsets, lens in ((c.offsets, [400, 300]), ([0, 1, 70], [100, 300]), ([10, 50, 60], [399, 10])):
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        c.views[0].seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.tiers[0].lens = np.array(lens)
        for _ in range(2):
            out.fill_(7.0)
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            got = out.cpu().numpy()
            c.check(got, offsets=offsets)
            assert (got[:offsets[0]] == 7.0).all() and (got[offsets[2]:] == 7.0).all()
            keep, c.q = c.q, last.cpu().numpy()
            c.check(one.cpu().numpy(), offsets=[0, 1, 2])
            c.q = keep


def test_another_stream_and_calls_at_once():
    torch, kvq = modules()
    cases = [Case(kvq, torch, [name], [[500, 300]], [40, 30], hq=4, hkv=2, seed=s) for s, name in enumerate(["cb4", "fp16", "fp8_int4"])]
    want = [c.run(kvq, torch) for c in cases]
    jobs = []
    for c in cases:
        q = torch.from_numpy(c.q).cuda()
        jobs.append((c, q, torch.empty_like(q), torch.tensor(c.offsets, dtype=torch.int32, device="cuda"),
                     torch.empty(kvq.kvq_chunk_workspace_size(c.views, 2, 70, 4), dtype=torch.uint8, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for c, q, out, off, ws, stream in jobs:
            kvq.kvq_chunk_attention(c.views, off, q, out, ws, stream=stream)
    torch.cuda.synchronize()
    for x, (_, _, out, *_) in zip(want, jobs):
        assert np.array_equal(out.cpu().numpy(), x)


def test_without_offsets_and_without_a_window():
    """One token a sequence by NULL offsets, and the decode form that sees everything: kvq_decode_attention's, rounded."""
    torch, kvq = modules()
    for name, d in (("fp8_int4", 128), ("cb4", 128), ("fp16", 64)):
        c = Case(kvq, torch, [name], [[700, 0, 1, 65, 300]], [1] * 5, hq=8, hkv=2, d=d, seed=11)
        q = torch.from_numpy(c.q).cuda()
        out = torch.empty_like(q)
        ws = torch.empty(kvq.kvq_chunk_workspace_size(c.views, 5, 5, 8), dtype=torch.uint8, device="cuda")
        kvq.kvq_chunk_attention(c.views, None, q, out, ws)
        assert np.array_equal(out.cpu().numpy(), c.run(kvq, torch))
        full = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        ws = torch.empty(kvq.kvq_decode_workspace_size(c.views, 5, 8), dtype=torch.uint8, device="cuda")
        kvq.kvq_decode_attention(c.views, q, full, ws)
        assert np.array_equal(c.run(kvq, torch, decode=True), full.half().cpu().numpy())


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (1, 2 ** 31 - 1), (2 ** 30, 5)])
def test_largest_windows(window, sinks):
    """Windows and sinks beyond any sequence, for chunks longer than theirs too."""
    torch, kvq = modules()
    for counts in ([30, 40], [1, 1]):
        c = Case(kvq, torch, ["cb4", "fp16"], [[200, 5], [20, 3]], counts, hq=2, hkv=1, window=window, sinks=sinks, seed=1)
        c.check(c.run(kvq, torch))
    c.check(c.run(kvq, torch, decode=True))


@pytest.mark.parametrize("d,hq", [(128, 2), (128, 16), (64, 2)])
def test_pools_beyond_four_gigabytes(d, hq):
    """Pages whose rows lie beyond 2^32 bytes of a pool: packed, unpacked, and under a window."""
    torch, kvq = modules()
    ps, hkv = 16, 2
    c = Case(kvq, torch, ["fp16"], [[300, 90]], [70, 9], hq=hq, hkv=hkv, d=d, window=200, sinks=3, seed=2)
    small = c.built.gpu[0]
    pages = 2 ** 32 // (ps * hkv * d * 2) + 1000
    far = kvq.PagedCache(d, hkv, pages, "fp16", "fp16", 0, 0, small.k_signs, small.v_signs, ps)
    n = small.num_pages
    far.k_rows[-n:], far.v_rows[-n:] = small.k_rows, small.v_rows
    want, one = c.run(kvq, torch), None
    c.views[0] = kvq.TierView(far, c.views[0].block_table + (pages - n), c.views[0].seq_lens)
    assert np.array_equal(c.run(kvq, torch), want)
    q = torch.from_numpy(c.q[[69, 78]]).cuda()
    got, ws = torch.empty_like(q), torch.empty(kvq.kvq_decode_window_workspace_size(c.views, 2, hq, 200, 3), dtype=torch.uint8, device="cuda")
    kvq.kvq_decode_attention_window(c.views, q, got, ws, 200, 3)
    keep, c.q = c.q, c.q[[69, 78]]
    c.check(got.cpu().numpy(), offsets=[0, 1, 2])
    c.q = keep


@pytest.mark.parametrize("name,count", [("cb4", 20), ("cb4", 300), ("cb32", 300), ("cb4+fp16", 300), ("cb4+fp16", 20)])
def test_values_of_very_different_sizes(name, count):
    """Values that grow and shrink by powers of two along the context, zero among them, under scores that favour the small ones:
    weights have to keep their precision whatever the values' norms."""
    torch, kvq = modules()

    def edit(tier, b, k, v):
        t = np.arange(len(v))
        v *= (2.0 ** ((t * 7) % 17 - 10.0))[:, None, None].astype(np.float16)
        v[::5] = 0
        k *= np.where(t % 5 == 0, 1.5, 0.7)[:, None, None].astype(np.float16)
    specs = name.split("+")
    lens = [[700]] if len(specs) == 1 else [[500], [200]]
    c = Case(kvq, torch, specs, lens, [count], hq=2, hkv=1, seed=12, edit=edit)
    c.check(c.run(kvq, torch), set(range(0, count, 11)))


def test_append_then_chunk_then_decode():
    """As a serving loop uses them: a prompt in chunks, turned and appended, attended under a window, then steps of one
    token; each against a call over the whole prompt."""
    torch, kvq = modules()
    rng = np.random.default_rng(0)
    d, hkv, hq, ps, total, window, sinks = 128, 2, 8, 16, 420, 96, 4
    ks, vs = kvq.kvq_make_signs(1, 0, hkv, d)
    rope = kvq.Rope(d, base=10000.0)
    x = torch.from_numpy(rng.standard_normal((total, hq + 2 * hkv, d)).astype(np.float16)).cuda()
    positions = torch.arange(total, dtype=torch.int32, device="cuda")

    def cache():
        return kvq.PagedCache(d, hkv, total // ps + 2, "fp8_e4m3", "int4_g32", 0, 0, ks, vs, ps)
    table = torch.from_numpy(rng.permutation(total // ps + 2)[None].astype(np.int32)).cuda()
    slots = (table[0].long()[positions.long() // ps] * ps + positions.long() % ps).to(torch.int32)

    def attend(c, first, last, one):
        q = torch.empty((last - first, hq, d), dtype=torch.float16, device="cuda")
        part = x[first:last]
        kvq.kvq_rope_append(c.struct, rope, positions[first:last], part[:, hq:hq + hkv], part[:, hq + hkv:], slots[first:last],
                            part[:, :hq], q)
        views = [kvq.TierView(c, table, torch.tensor([last], dtype=torch.int32, device="cuda"))]
        out = torch.empty_like(q)
        if one:
            ws = torch.empty(kvq.kvq_decode_window_workspace_size(views, 1, hq, window, sinks), dtype=torch.uint8, device="cuda")
            kvq.kvq_decode_attention_window(views, q, out, ws, window, sinks)
        else:
            ws = torch.empty(kvq.kvq_chunk_workspace_size(views, 1, last - first, hq, window, sinks), dtype=torch.uint8, device="cuda")
            kvq.kvq_chunk_attention(views, torch.tensor([0, last - first], dtype=torch.int32, device="cuda"), q, out, ws, window, sinks)
        return out
    whole = attend(cache(), 0, total, False).float()
    c = cache()
    parts = [attend(c, a, b, False) for a, b in ((0, 200), (200, 201), (201, 417))] + [attend(c, t, t + 1, True) for t in range(417, total)]
    got = torch.cat(parts).float()
    # each side is within 2^-9 of the exact result (2-norm), and so of the other within twice that
    assert float((got - whole).norm() / whole.norm()) <= 2.0 ** -8
