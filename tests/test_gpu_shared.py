"""GPU parity of kvq_decode_attention_shared against the float64 oracle, on bytes that the
oracle wrote.

Tolerance, derived before the first run, u = 2^-11 (half an ulp of fp16, relative).
A score: the rotated queries are rounded once and the decoded keys at most twice (table entry,
product with the norm), so with S_t = sum_i |q~_i| |k~_ti| / sqrt(D) a score is off by at most
3 u S_t (1 + 2^-9) and float32 accumulation (2^-15 S_t covers 128 additions); a weight by the
factor e^d, d = max_t of that, twice (numerator and denominator).  The weights themselves are
rounded to fp16 in the numerator (u, or 2^-25 absolute where they fall below 2^-14 of the running
maximum, which itself is within 2^8 of the row's: 2^-17 of the largest weight at most, summed
over L tokens L 2^-17 ... taken exactly as 2^-25 L max|V| / sum of weights >= 1), the decoded
values at most twice (2 u of |v~|, spread by the inverse rotation: |v~|'s 2-norm is |v|'s, and a
coordinate of the result sees at most the 2-norm of the rounding errors, 2 u |v|_2), and the
output once.  The bound is worst-case; independent roundings add in squares, so the 2-norm
over all outputs is held to 2^-9 of the outputs' besides: scores off by about u sqrt(3) (unit
variance), weights u, values u sqrt(2), output u: in squares under 3 u, and 4 u allowed."""
import math

import numpy as np
import pytest

import workloads as W
from oracle import attention as oatt
from oracle import rotation as orot
from oracle import shared as oshared
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -11

SPECS = {
    "fp16": W.Tier("fp16", "fp16"),
    "fp8_int4": W.Tier("fp8_e4m3", "int4_g32"),
    "fp8_fp16": W.Tier("fp8_e4m3", "fp16"),
    "cb4": W.Tier("codebook", "codebook", 4, 4),
    "cb32": W.Tier("codebook", "codebook", 3, 2),
    "cb23": W.Tier("codebook", "codebook", 2, 3, codebook="uniform"),
    "qjl": W.Tier("codebook_qjl", "codebook", 3, 4),
    "outlier": W.Tier("codebook_outlier", "codebook", 4, 4),
}


class Case:
    def __init__(self, kvq, torch, specs, prefix_lens, offsets, own_specs, own_lens, hq, hkv, d=128, ps=16, seed=0,
                 spread=1.0):
        """specs / own_specs: tier names; prefix_lens: per tier, a length per group; own_lens: per
        tier, a length per sequence."""
        rng = np.random.default_rng([seed, hq, hkv, d, ps])
        self.batch = len(own_lens[0]) if own_specs else offsets[-1]
        n = max(self.batch, len(offsets) - 1, 1)
        kv = []
        for lens in list(prefix_lens) + list(own_lens):
            lens = list(lens) + [0] * (n - len(lens))
            kv.append([tuple((rng.standard_normal((L, hkv, d)) * s).astype(np.float16) for s in (spread, 1.0)) for L in lens])
        ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
        tiers = [SPECS[s] for s in list(specs) + list(own_specs)]
        proj = rng.standard_normal((128, d)).astype(np.float32)
        outl = np.stack([rng.choice(d, 8, replace=False) for _ in range(hkv)]).astype(np.int32)
        self.built = gu.build_exact(kvq, torch, tiers, kv, ks, vs, ps, shuffle_seed=seed + 1, k_qjl=proj, k_outl=outl)
        first = self.built.gpu[0].struct
        for c in self.built.gpu[1:]:  # one projection, as the calls want it
            c.struct.k_signs, c.struct.v_signs = first.k_signs, first.v_signs
            if c.struct.k_qjl and first.k_qjl:
                c.struct.k_qjl = first.k_qjl
        m = len(specs)
        self.prefix, self.own = self.built.views[:m], self.built.views[m:]
        self.offsets = list(offsets)
        ora = self.built.ora
        for t in ora[m:]:
            t.block_table, t.lens = t.block_table[:self.batch], t.lens[:self.batch]
        self.tiers = oshared.as_tiers(ora[:m], self.offsets, ora[m:], self.batch)
        self.q = rng.standard_normal((self.batch, hq, d)).astype(np.float16)
        self.hq, self.hkv, self.d = hq, hkv, d

    def run(self, kvq, torch, q=None, out=None, ws=None):
        q = torch.from_numpy(self.q).cuda() if q is None else q
        need = kvq.kvq_decode_shared_workspace_size(self.prefix, self.offsets, self.own, self.batch, self.hq)
        out_buf, out = gu.guarded_empty(torch, tuple(q.shape), torch.float16)
        ws_buf, ws = gu.guarded_empty(torch, (need,), torch.uint8)
        ws.fill_(0xFF)  # what a workspace holds does not matter
        status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        kvq.kvq_decode_attention_shared(self.prefix, self.offsets, self.own, q, out, ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0, f"device error bits {int(status.item())}"
        gu.assert_guards(out_buf, out)
        gu.assert_guards(ws_buf, ws)
        return out.cpu().numpy()

    def check(self, got, heads=None):
        grp = self.hq // self.hkv
        sum_off = sum_size = 0.0
        for b in range(self.batch):
            for h in range(self.hq):
                if heads is not None and (b, h) not in heads:
                    continue
                keys, values = oatt.dequantised_kv(self.tiers, b, h // grp)
                g = got[b, h].astype(np.float64)
                if keys is None:
                    assert not g.any()
                    continue
                q = self.q[b, h].astype(np.float64)
                extra = oatt.sketch_terms(self.tiers, b, h // grp, q)
                s = (keys @ q + extra) / math.sqrt(self.d)
                w = np.exp(s - s.max())
                w /= w.sum()
                want = w @ values
                signs = self.built.k_signs[h // grp]
                qr, kr = np.abs(orot.rotate(q, signs)), np.abs(orot.rotate(keys, signs))
                off = float(np.max((3 * U * (1 + 2.0 ** -9) + 2.0 ** -15) * (kr @ qr) / math.sqrt(self.d)))
                size = np.linalg.norm(values, axis=-1)
                tol = (2 * math.expm1(off) + U) * (w @ np.abs(values)) + 2 * U * (w @ size)
                tol = (tol + 2.0 ** -25 * len(w) * np.max(np.abs(values))) * (1 + 2.0 ** -9) + U * np.abs(want) + 2.0 ** -25
                bad = np.abs(g - want) > tol
                assert not bad.any(), f"({b}, {h}): {int(bad.sum())} off, worst {np.max(np.abs(g - want) / tol)}"
                sum_off += float(np.sum((g - want) ** 2))
                sum_size += float(np.sum(want ** 2))
        rel = math.sqrt(sum_off / max(sum_size, 1e-300))
        assert sum_size == 0 or rel <= 2.0 ** -9, f"relative error {rel}"


def modules():
    return gu.torch_cuda(), gu.kvq_module()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 1000])
def test_lengths(length):
    """One prefix of every awkward length, a few sequences of one token each."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16"], [[length]], [0, 3], ["fp16"], [[1, 1, 1]], hq=4, hkv=2, seed=length)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name", ["fp16", "fp8_int4", "fp8_fp16", "cb4", "cb32", "cb23"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_formats_and_groups(name, group):
    torch, kvq = modules()
    own = [[0, 5, 33, 16, 1]]
    c = Case(kvq, torch, [name], [[700]], [0, 5], [name], own, hq=2 * group, hkv=2, seed=group)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("batch,group", [(16, 8), (17, 8), (31, 8), (32, 8), (33, 8), (70, 4), (130, 1), (300, 1)])
def test_row_blocks(batch, group):
    """Rows around the sizes of an accumulator (128) and of an item (256), more than one item."""
    torch, kvq = modules()
    rng = np.random.default_rng(batch)
    c = Case(kvq, torch, ["fp8_int4"], [[391]], [0, batch], ["fp8_int4"], [rng.integers(0, 9, batch)], hq=group, hkv=1,
             seed=batch)
    heads = {(b, h) for b in list(range(0, batch, 7)) + [batch - 1, batch - 2] for h in range(group)}
    c.check(c.run(kvq, torch), heads)


@pytest.mark.parametrize("ps", [1, 5, 12, 16, 24, 64])
def test_page_sizes(ps):
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb4"], [[333]], [0, 4], ["cb4"], [[3, 0, 40, 7]], hq=4, hkv=2, ps=ps, seed=ps)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("name", ["cb4", "cb32", "fp8_int4", "fp16"])
@pytest.mark.parametrize("batch,group", [(5, 1), (40, 4)])
def test_long_chunks(name, batch, group):
    """Work items of ten tiles and more, both ways of sharing them between the softmax groups: the
    rings of tiles, rows and norms go round several times."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[20000]], [0, batch], [name], [[3] * batch], hq=8 * group, hkv=8, seed=batch)
    heads = {(b, h) for b, h in ((0, 0), (1, group), (batch - 1, 8 * group - 1), (batch // 2, 5 * group))}
    c.check(c.run(kvq, torch), heads)


def test_ragged_groups():
    """Groups of different sizes and lengths, one empty, one of length 0, sequences before the
    first group and behind the last, a sequence without a token."""
    torch, kvq = modules()
    offsets = [2, 5, 5, 40, 41, 43]
    own = np.random.default_rng(3).integers(0, 50, 45)
    own[0], own[41], own[44] = 0, 0, 0  # 0: no group and nothing of its own
    c = Case(kvq, torch, ["cb4"], [[300, 77, 1500, 0, 129]], offsets, ["cb4"], [own], hq=8, hkv=2, seed=5)
    got = c.run(kvq, torch)
    assert not got[0].any() and not got[44].any()
    c.check(got, {(b, h) for b in (0, 1, 2, 4, 5, 20, 39, 40, 41, 42, 43, 44) for h in range(8)})


def test_most_groups():
    """As many groups as a call takes, most of one sequence or none."""
    torch, kvq = modules()
    n = kvq.MAX_PREFIX_GROUPS
    rng = np.random.default_rng(17)
    offsets = [0] + np.cumsum(rng.integers(0, 3, n)).tolist()
    lens = rng.integers(0, 200, n)
    c = Case(kvq, torch, ["fp8_int4"], [lens], offsets, ["fp8_int4"], [rng.integers(0, 5, offsets[-1] + 2)], hq=2, hkv=1,
             seed=17)
    heads = {(b, h) for b in list(range(0, c.batch, 11)) + [offsets[-1] - 1, c.batch - 1] for h in range(2)}
    c.check(c.run(kvq, torch), heads)


def test_tiers_of_the_prefix_and_of_the_sequences():
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16", "fp8_int4"], [[100, 0], [900, 260]], [0, 4, 7], ["fp8_int4", "fp16"],
             [[20, 0, 3, 200, 1, 7, 0], [0, 16, 16, 16, 2, 0, 0]], hq=8, hkv=2, seed=8)
    c.check(c.run(kvq, torch))


def test_codebook_and_other_tiers_of_one_prefix():
    """Two kinds of prefix tier: a launch each."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb32", "fp16"], [[700, 90], [64, 16]], [0, 4, 7], ["cb4"], [[20, 0, 3, 200, 1, 7, 0]], hq=8,
             hkv=2, seed=15)
    c.check(c.run(kvq, torch))


def test_no_tokens_of_their_own():
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb32"], [[450]], [0, 6], [], [], hq=4, hkv=2, seed=9)
    c.check(c.run(kvq, torch))


@pytest.mark.parametrize("spread", [8.0, 40.0])
def test_large_scores(spread):
    """Keys large enough that running maxima move by far more than the rescaling threshold."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16"], [[1200]], [0, 20], ["fp16"], [[4] * 20], hq=8, hkv=1, seed=10, spread=spread)
    got = c.run(kvq, torch)
    grp = c.hq // c.hkv
    # scores of this size leave no worst-case bound to speak of; a score's float32 and fp16
    # roundings, independent, give it 2 u sqrt(sum (q~ k~)^2 / D) of noise (three sigma), and the
    # weights that factor: compared where the softmax is not decided by less than that
    for b in range(0, c.batch, 5):
        for h in range(c.hq):
            keys, values = oatt.dequantised_kv(c.tiers, b, h // grp)
            q = c.q[b, h].astype(np.float64)
            s = keys @ q / math.sqrt(c.d)
            w = np.exp(s - s.max())
            w /= w.sum()
            signs = c.built.k_signs[0]
            noise = 2 * U * np.sqrt((orot.rotate(keys, signs) ** 2) @ (orot.rotate(q, signs) ** 2)) / math.sqrt(c.d)
            d = 3 * float(np.max(noise))
            tol = 2 * math.expm1(d) * (w @ np.abs(values - w @ values)) + 8 * U * (w @ np.linalg.norm(values, axis=-1))
            assert np.all(np.abs(got[b, h] - w @ values) <= tol + 2.0 ** -20)


@pytest.mark.parametrize("name,d", [("qjl", 128), ("outlier", 128), ("outlier", 256), ("cb4", 64), ("fp8_int4", 64),
                                    ("cb4", 256), ("fp16", 256)])
def test_prefix_as_a_tier_of_every_sequence(name, d):
    """Formats and sizes the prefix kernel is not built for."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[200, 37]], [1, 3, 5], [name], [[5, 0, 20, 1, 0, 3]], hq=4, hkv=2, d=d, seed=d)
    c.check(c.run(kvq, torch))


def test_same_result_as_plain_decode():
    """The prefix as an ordinary tier of every sequence, by kvq_decode_attention: the same
    function, within the bounds of both (its own is far smaller)."""
    torch, kvq = modules()
    batch = 24
    c = Case(kvq, torch, ["fp8_int4"], [[2000]], [0, batch], ["fp16"], [[10] * batch], hq=32, hkv=8, seed=12)
    got = c.run(kvq, torch).astype(np.float64)
    pre = c.prefix[0]
    views = [kvq.TierView(pre.cache, pre.block_table[:1].expand(batch, -1).contiguous(),
                          pre.seq_lens[:1].expand(batch).contiguous()), c.own[0]]
    want = gu.gpu_decode(kvq, torch, views, c.q).astype(np.float64)
    assert np.linalg.norm(got - want) <= 2.0 ** -9 * np.linalg.norm(want)


def test_deterministic_replays_and_two_graphs():
    """Two captured graphs with a workspace each, an eager call on another stream; lengths that
    grow between replays are read when the graph runs."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb4"], [[640]], [0, 9], ["cb4"], [[30] * 9], hq=8, hkv=2, seed=13)
    q = torch.from_numpy(c.q).cuda()
    need = kvq.kvq_decode_shared_workspace_size(c.prefix, c.offsets, c.own, 9, 8)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)]
    outs = [torch.zeros_like(q) for _ in range(3)]
    call = lambda i: kvq.kvq_decode_attention_shared(c.prefix, c.offsets, c.own, q, outs[i], ws[i])  # noqa: E731
    call(0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for lens in ([30] * 9, list(range(20, 29))):
        c.own[0].seq_lens[:9].copy_(torch.tensor(lens, dtype=torch.int32))
        c.tiers[-1].lens[:] = lens
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for g in graphs:
            g.replay()
        with torch.cuda.stream(side):
            call(2)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        c.check(outs[0].cpu().numpy())


def test_bad_lengths_and_pages_are_reported():
    """What only the device can see: a length beyond the table, a page outside the pool.  Checked on
    the CPU first (tests/test_index_checks.py): no read is made through either."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["cb4"], [[300]], [0, 3], ["cb4"], [[4, 4, 4]], hq=2, hkv=2, seed=14)
    q, out = torch.from_numpy(c.q).cuda(), torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size(c.prefix, c.offsets, c.own, 3, 2), dtype=torch.uint8,
                     device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def bits():
        kvq.kvq_decode_attention_shared(c.prefix, c.offsets, c.own, q, out, ws, status)
        return int(status.item())

    assert bits() == 0
    table, lens = c.prefix[0].block_table, c.prefix[0].seq_lens
    keep = table.clone()
    for bad in (-1, c.built.gpu[0].num_pages, 2 ** 31 - 1):
        table[0, 3] = bad
        assert bits() == kvq.DEVERR_PAGE_INDEX
        table.copy_(keep)
    for bad in (-5, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        lens[0] = bad
        assert bits() & kvq.DEVERR_SEQ_LEN
    lens[0] = 300
    assert bits() == 0
    c.check(out.cpu().numpy())


def test_one_token_against_a_long_tail():
    """A token that outweighs each of 131071 others 2^25.5 times: together they hold 0.3% of the
    weight, and with values eight times as large 2% of the output.  Half a step of fp16 against a
    weight of 1 would lose them all; with a largest weight of 4 each is kept to 2^-25 / 4 of it,
    together 2^17 2^-27 8 = 2^-7 of the large token's value, beside 2^-9 (2-norm) for the other
    roundings (losing them all would be 2.2%).  The others are one page, 8191 times in the table."""
    torch, kvq = modules()
    d, ps, hkv, group, batch, pages = 128, 16, 150, 8, 16, 8192
    rng = np.random.default_rng(15)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    cache = kvq.PagedCache(d, hkv, 2, "fp16", "fp16", 0, 0, ks, vs, ps)
    u = rng.standard_normal((hkv, d))
    u /= np.linalg.norm(u, axis=-1, keepdims=True)
    gap = 25.5 * math.log(2.0)  # nats, between scores of the queries below
    length = 12.0  # of the queries
    k = np.repeat((-0.5 * gap * math.sqrt(d) / length * u)[None], 2 * ps, 0).astype(np.float16)
    k[5] = (0.5 * gap * math.sqrt(d) / length * u).astype(np.float16)
    v = np.repeat(8 * rng.standard_normal((1, hkv, d)), 2 * ps, 0).astype(np.float16)
    v[5] = rng.standard_normal((hkv, d)).astype(np.float16)
    slots = torch.arange(2 * ps, dtype=torch.int32, device="cuda")
    cache.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots)
    table = torch.ones(1, pages, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    view = kvq.TierView(cache, table, torch.tensor([pages * ps], dtype=torch.int32, device="cuda"))
    q = np.repeat((length * u).astype(np.float16), group, 0)[None].repeat(batch, 0)
    qd = torch.from_numpy(np.ascontiguousarray(q)).cuda()
    out = torch.empty_like(qd)
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size([view], [0, batch], None, batch, hkv * group),
                     dtype=torch.uint8, device="cuda")
    kvq.kvq_decode_attention_shared([view], [0, batch], None, qd, out, ws)
    got = out.cpu().numpy().astype(np.float64)
    # what the cache holds, read back (each vector rounded once more: 2^-11 of it)
    kb, vb = (torch.empty(2 * ps, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    kvq.kvq_dequantize(cache.struct, slots, kb, vb)
    kb, vb = kb.cpu().numpy().astype(np.float64), vb.cpu().numpy().astype(np.float64)
    for h in range(0, hkv, 7):
        s = kb[:, h] @ q[0, h * group].astype(np.float64) / math.sqrt(d)
        count = np.array([1.0] * ps + [float(pages - 1)] * ps)  # page 1's tokens, 8191 times
        p = count * np.exp(s - s.max())
        tail = 1.0 - p[5] / p.sum()
        assert 1e-3 < tail < 6e-3, tail
        want = (p / p.sum()) @ vb[:, h]
        for b in (0, batch - 1):
            off = np.linalg.norm(got[b, h * group:(h + 1) * group] - want, axis=-1)
            # scores near +-8.8 nats: queries and keys rounded, together 4 u of a score at most, move the
            # tail's share by 2 * 8.9 * 4 u = 3.5% of itself, 0.1% of the output
            limit = (2.0 ** -9 + 2.0 ** -7) * np.linalg.norm(vb[5, h]) + 0.035 * tail * np.linalg.norm(vb[0, h])
            assert np.all(off <= limit), (off.max(), limit, tail * np.linalg.norm(vb[0, h]))


def test_a_tier_without_pages_is_reported():
    """A prefix tier whose table has no columns: a length above zero is out of range, and the other
    tiers are attended as if it were not there."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp16", "fp16"], [[300], [0]], [0, 3], ["fp16"], [[4, 4, 4]], hq=2, hkv=2, seed=16)
    empty = kvq.TierView(c.prefix[1].cache, torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                         torch.zeros(1, dtype=torch.int32, device="cuda"))
    q, out = torch.from_numpy(c.q).cuda(), torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    pre = [c.prefix[0], empty]
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size(pre, [0, 3], c.own, 3, 2), dtype=torch.uint8, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    for length, bits in ((0, 0), (1, kvq.DEVERR_SEQ_LEN), (-1, kvq.DEVERR_SEQ_LEN), (0, 0)):
        empty.seq_lens.fill_(length)
        kvq.kvq_decode_attention_shared(pre, [0, 3], c.own, q, out, ws, status)
        assert int(status.item()) == bits
        c.check(out.cpu().numpy())


def test_status_of_many_sequences():
    """A length out of range is found wherever it stands among 2000 sequences."""
    torch, kvq = modules()
    batch = 2000
    c = Case(kvq, torch, ["fp8_int4"], [[40]], [0, batch], ["fp8_int4"], [[1] * batch], hq=1, hkv=1, seed=17)
    q, out = torch.from_numpy(c.q).cuda(), torch.empty(c.q.shape, dtype=torch.float16, device="cuda")
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size(c.prefix, c.offsets, c.own, batch, 1), dtype=torch.uint8,
                     device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    lens = c.own[0].seq_lens
    for at in (None, 0, 777, batch - 1):
        if at is not None:
            lens[at] = -3
        kvq.kvq_decode_attention_shared(c.prefix, c.offsets, c.own, q, out, ws, status)
        assert int(status.item()) == (0 if at is None else kvq.DEVERR_SEQ_LEN)
        if at is not None:
            lens[at] = 1


@pytest.mark.parametrize("power", [-9, 7])
@pytest.mark.parametrize("name", ["cb4", "cb23"])
def test_codebooks_of_any_size(name, power):
    """Centroids times a power of two, norms over it: the same output, to the bit."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[500]], [0, 3], [], [], hq=8, hkv=2, seed=18)
    want = c.run(kvq, torch)
    c.check(want)
    cache = c.built.gpu[0]
    for cent, aux in ((cache.k_centroids, cache.k_aux), (cache.v_centroids, cache.v_aux)):
        cent.mul_(2.0 ** power)
        aux.mul_(2.0 ** -power)
    assert np.array_equal(c.run(kvq, torch), want)


@pytest.mark.parametrize("name,batch,group", [("cb4", 6, 4), ("fp8_int4", 40, 8)])
def test_a_query_that_is_not_finite_stays_in_its_row(name, batch, group):
    """A NaN or an infinity in one query: its own output is NaN, every other row as ever."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[900]], [0, batch], [name], [[3] * batch], hq=2 * group, hkv=2, seed=19)
    q = c.q.copy()
    bad = {(1, 0): np.nan, (batch - 1, 2 * group - 1): np.inf}
    for (b, h), v in bad.items():
        q[b, h, 5] = v
    out = c.run(kvq, torch, torch.from_numpy(q).cuda())
    for b, h in bad:
        assert np.isnan(out[b, h]).all()
    heads = {(b, h) for b in (0, 1, batch // 2, batch - 1) for h in range(2 * group)} - set(bad)
    c.check(out, heads)


@pytest.mark.parametrize("name", ["fp16", "cb4"])
@pytest.mark.parametrize("length", [1, 130, 261])
def test_what_lies_behind_the_prefix_is_not_read(name, length):
    """NaN in every slot of the pool that holds no token of the prefix, its last page's among them."""
    torch, kvq = modules()
    c = Case(kvq, torch, [name], [[length]], [0, 3], [], [], hq=8, hkv=2, seed=length)
    want = c.run(kvq, torch)
    c.check(want)
    cache, table = c.built.gpu[0], c.prefix[0].block_table.cpu().numpy()[0]
    t = np.arange(length)
    held = table[t // 16] * 16 + t % 16
    free = np.setdiff1d(np.arange(cache.num_pages * 16), held)
    pages, offs = (torch.from_numpy(x).cuda() for x in (free // 16, free % 16))
    sides = (cache.k_rows, cache.v_rows) if name == "fp16" else (cache.k_aux, cache.v_aux)
    for a in sides:
        if a.dtype == torch.float16:
            a[pages, :, offs] = float("nan")
        else:
            a[pages, :, offs] = 0x7E  # bytes of fp16 NaN
    assert np.array_equal(c.run(kvq, torch), want)


def test_one_page_many_times():
    """A block table that names one page again and again: attention over copies of its tokens."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[16]], [0, 5], [], [], hq=8, hkv=2, seed=20)
    want = c.run(kvq, torch).astype(np.float64)
    c.check(want)
    view = c.prefix[0]
    many = kvq.TierView(view.cache, view.block_table[:, :1].expand(-1, 300).contiguous(),
                        torch.full_like(view.seq_lens, 4800))
    q = torch.from_numpy(c.q).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size([many], [0, 5], None, 5, 8), dtype=torch.uint8, device="cuda")
    kvq.kvq_decode_attention_shared([many], [0, 5], None, q, out, ws)
    got = out.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= 2.0 ** -9 * np.linalg.norm(want)
