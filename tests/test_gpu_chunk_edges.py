"""GPU tests of kvq_chunk_attention and kvq_decode_attention_window at what no query sees: block-table
entries, vectors and scales of tokens outside the windows and sinks of a call must not reach its
results or its status.  Results are held to the bounds of test_gpu_chunk (its docstring derives
them), where they are looked at for the sequence in question alone."""
import numpy as np
import pytest

from oracle import chunk as ochunk
from tests.test_gpu_chunk import Case, modules

pytestmark = pytest.mark.gpu


def unseen_entries(c, counts):
    """Per tier [batch, pages]: entries of the block table that hold no token that a query sees."""
    out = []
    for i, tier in enumerate(c.tiers):
        free = np.ones(tier.block_table.shape, dtype=bool)
        for b, count in enumerate(counts):
            length, base = (sum(int(t.lens[b]) for t in tiers) for tiers in (c.tiers, c.tiers[:i]))
            seen = np.zeros(length, dtype=bool)
            for p in range(length - count, length):
                seen |= ochunk.sees(p, length, c.window, c.sinks)
            for t in np.flatnonzero(seen[base:base + int(tier.lens[b])]):
                free[b, t // tier.page_size] = False
        out.append(free)
    return out


# one sequence of ordinary tokens and one of large ones, whose pages stand in for those that are not seen
def two_sequences(name, d, hq, lens, counts, window, sinks, ps=16, hkv=1):
    torch, kvq = modules()

    def edit(tier, b, k, v):
        v *= np.float16(2.0 ** 11 if b else 2.0 ** -3)
    specs = name.split("+")
    return torch, kvq, Case(kvq, torch, specs, [[n, n] for n in lens], [counts, counts], hq=hq, hkv=hkv, d=d, ps=ps, window=window,
                            sinks=sinks, seed=window + 3 * sinks, edit=edit)


def give_away(torch, c, free, other):
    """Unseen entries of both sequences: outside the pool, or (of the first) the second's pages."""
    for view, f, tier in zip(c.views, free, c.tiers):
        table = view.block_table.cpu().numpy()
        if other == "outside":
            table[f] = np.resize([-1, 1 << 30, -(1 << 31)], int(f.sum()))
        else:
            pages = tier.block_table[1, :max(1, (int(tier.lens[1]) + tier.page_size - 1) // tier.page_size)]
            table[0, f[0]] = np.resize(pages, int(f[0].sum()))
        view.block_table.copy_(torch.from_numpy(table))


def check_both(c, got, count):
    """Each sequence by itself: the larger's outputs do not stand in for the smaller's."""
    for b in range(2):
        c.check(got, set(range(b * count, (b + 1) * count)))


# (page size 24: pages and tiles end at different tokens)
WINDOWS = [(1, 0), (33, 0), (40, 4), (100, 20), (130, 140), (257, 3)]
PACKED = [("fp16", 128, 2, 20), ("fp8_int4", 128, 2, 20), ("fp8_fp16", 128, 1, 150), ("cb4", 128, 2, 20), ("cb32", 128, 1, 150)]
UNPACKED = [("fp16", 128, 8, 120), ("fp8_int4", 128, 8, 120), ("cb4", 128, 8, 120), ("cb32", 256, 2, 20), ("cb4", 64, 1, 9),
            ("fp16", 64, 2, 150), ("qjl", 128, 1, 7), ("outlier", 128, 2, 7), ("fp8_int4", 256, 1, 20)]


@pytest.mark.parametrize("name,d,hq,count", PACKED)
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("other", ["outside", "large"])
def test_packed_pages_that_no_query_sees(name, d, hq, count, window, sinks, other):
    for ps in (16, 24):
        torch, kvq, c = two_sequences(name, d, hq, [700], count, window, sinks, ps)
        give_away(torch, c, unseen_entries(c, [count, count]), other)
        check_both(c, c.run(kvq, torch), count)


@pytest.mark.parametrize("specs,lens,hq,count", [("fp8_int4+fp16", [500, 200], 2, 20), ("cb4+fp16", [333, 90], 2, 33),
                                                 ("cb32+cb4+fp8_int4+fp16", [130, 101, 203, 60], 1, 9)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("other", ["outside", "large"])
def test_packed_pages_of_tiers_that_no_query_sees(specs, lens, hq, count, window, sinks, other):
    torch, kvq, c = two_sequences(specs, 128, hq, lens, count, window, sinks)
    give_away(torch, c, unseen_entries(c, [count, count]), other)
    check_both(c, c.run(kvq, torch), count)


@pytest.mark.parametrize("name,d,hq,count", UNPACKED)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_unpacked_pages_that_no_query_sees(name, d, hq, count, window, sinks):
    for ps in (16,) if name in ("qjl", "outlier") else (16, 24):  # (keys with a sketch or outliers: 16 only)
        torch, kvq, c = two_sequences(name, d, hq, [700], count, window, sinks, ps)
        give_away(torch, c, unseen_entries(c, [count, count]), "outside")
        check_both(c, c.run(kvq, torch), count)


@pytest.mark.parametrize("specs,lens,hq,count", [("fp8_int4+fp16", [500, 200], 8, 100), ("cb4+fp16", [333, 90], 8, 80),
                                                 ("cb32+cb4+fp8_int4+fp16", [130, 101, 203, 60], 8, 70)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_unpacked_pages_of_tiers_that_no_query_sees(specs, lens, hq, count, window, sinks):
    torch, kvq, c = two_sequences(specs, 128, hq, lens, count, window, sinks)
    give_away(torch, c, unseen_entries(c, [count, count]), "outside")
    check_both(c, c.run(kvq, torch), count)


@pytest.mark.parametrize("name,d,hq,lens", [("fp16", 128, 2, [300, 200]), ("fp8_int4", 128, 8, [301, 200]), ("cb4", 128, 1, [303, 100]),
                                            ("cb4", 128, 4, [303, 100]), ("cb32", 256, 2, [310, 77]), ("fp16", 64, 2, [297, 64]),
                                            ("qjl", 128, 1, [301, 64]), ("outlier", 128, 2, [301, 64])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (40, 4), (50, 300), (64, 17), (210, 5)])
@pytest.mark.parametrize("other", ["outside", "large"])
def test_decode_window_pages_that_the_query_does_not_see(name, d, hq, lens, window, sinks, other):
    """Also of a tier whose last page is not full and ends before the window."""
    for specs in (name, name + "+fp16"):
        for ps in (16,) if name in ("qjl", "outlier") else (16, 24):  # (keys with a sketch or outliers: 16 only)
            torch, kvq, c = two_sequences(specs, d, hq, lens[:specs.count("+") + 1], 1, window, sinks, ps)
            give_away(torch, c, unseen_entries(c, [1, 1]), other)
            check_both(c, c.run(kvq, torch, decode=True), 1)


@pytest.mark.parametrize("name,d,hq,count", [u for u in UNPACKED if u[0] not in ("fp16", "fp8_int4")])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_large_values_that_no_query_sees(name, d, hq, count, window, sinks):
    """Finite ones, on pages of another sequence, set no scale of those that are seen."""
    torch, kvq, c = two_sequences(name, d, hq, [700], count, window, sinks)
    give_away(torch, c, unseen_entries(c, [count, count]), "large")
    check_both(c, c.run(kvq, torch), count)


def early_case(specs, lens, count, hq, d, early, late):
    """Early tokens (400 of the first tier) with values of another size than all the others, seen, with next to no weight."""
    torch, kvq = modules()

    def edit(tier, b, k, v):
        old = np.arange(len(v)) < (400 if tier == 0 else 0)
        v *= np.where(old, early, late)[:, None, None].astype(np.float16)
        k[old] = np.float16(-4.0)
    c = Case(kvq, torch, specs.split("+"), [[n] for n in lens], [count], hq=hq, hkv=1, d=d, seed=1, edit=edit)
    c.q = (1.0 + 0.25 * np.random.default_rng(2).standard_normal(c.q.shape)).astype(np.float16)
    c.check(c.run(kvq, torch), set(range(0, count, 7)))


SIZES = [("cb4+fp16", [400, 300]), ("cb32+fp16", [400, 300]), ("cb4+fp8_int4", [400, 300]), ("cb4", [700]), ("cb32", [700])]
EARLY, LATE = [2.0 ** -17, 2.0 ** -12, 1.0, 2.0 ** 11], [2.0 ** -8, 8.0]


@pytest.mark.parametrize("specs,lens", SIZES)
@pytest.mark.parametrize("count,hq,d", [(120, 8, 128), (120, 8, 64), (20, 2, 256)])
@pytest.mark.parametrize("early", EARLY)
@pytest.mark.parametrize("late", LATE)
def test_values_of_early_tokens_set_no_scale_of_unpacked_ones(specs, lens, count, hq, d, early, late):
    early_case(specs, lens, count, hq, d, early, late)


@pytest.mark.parametrize("specs,lens", SIZES)
@pytest.mark.parametrize("count", [20, 300])
@pytest.mark.parametrize("early", EARLY)
@pytest.mark.parametrize("late", LATE)
def test_values_of_early_tokens_set_no_scale_of_packed_ones(specs, lens, count, early, late):
    early_case(specs, lens, count, 1, 128, early, late)


@pytest.mark.parametrize("d,hq,count", [(128, 8, 120), (64, 1, 5), (256, 1, 5), (128, 1, 5)])
def test_scales_of_other_sequences_pages_are_not_reported(d, hq, count):
    """INT4 scales that leave fp16, on the pool's first page, which holds no token of the call's sequences."""
    torch, kvq = modules()
    c = Case(kvq, torch, ["fp8_int4"], [[300, 77]], [count, 3], hq=hq, hkv=1, d=d, seed=3)
    cache, view, tier = c.built.gpu[0], c.views[0], c.tiers[0]
    held = np.zeros(cache.num_pages, dtype=bool)
    for b, n in enumerate(tier.lens):
        held[tier.block_table[b, :(int(n) + 15) // 16]] = True
    if held[0]:
        free = int(np.flatnonzero(~held)[0])
        for x in (cache.k_rows, cache.v_rows, cache.v_aux):
            x[free] = x[0]
        view.block_table[view.block_table == 0] = free
    cache.v_aux[0] = 60000.0
    c.check(c.run(kvq, torch))
