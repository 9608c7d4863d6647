"""Pins of the oracle's chunk attention: its last query is the decode query, a mask drawn by hand, and a sequence
cut short."""
import numpy as np
import pytest

from oracle import attention as oatt
from oracle import cache as oc
from oracle import chunk


def tier(rng, lens, hkv=2, d=64, ps=4):
    signs = np.where(rng.random((hkv, d)) < 0.5, -1, 1).astype(np.int8)
    per = [(n + ps - 1) // ps for n in lens]
    table = np.zeros((len(lens), max(1, max(per))), dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = np.arange(at, at + n)
        at += n
    sides = [oc.new_side("fp16", 0, None, None, signs, max(1, at), hkv, ps, d) for _ in range(2)]
    for b, n in enumerate(lens):
        t = np.arange(n)
        for side in sides:
            oc.write(side, table[b, t // ps] * ps + t % ps, rng.standard_normal((n, hkv, d)).astype(np.float16), ps)
    return oatt.TierState(sides[0], sides[1], table, np.array(lens), ps)


def test_sees_by_hand():
    rows = [chunk.sees(p, 7, 3, 2).astype(int).tolist() for p in (-1, 0, 2, 4, 6)]
    assert rows == [[0] * 7, [1, 0, 0, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0], [1, 1, 0, 0, 1, 1, 1]]
    assert chunk.sees(3, 6).tolist() == [True] * 4 + [False] * 2


def test_last_query_is_the_decode_query():
    rng = np.random.default_rng(1)
    t = tier(rng, [9, 5])
    q = rng.standard_normal((6, 4, 64)).astype(np.float16)
    got = chunk.chunk_attention(q, [t], [0, 4, 6])
    want = oatt.decode_attention(q[[3, 5]], [t])
    assert np.allclose(got[[3, 5]], want, rtol=0, atol=1e-6)  # (float32 results)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 2), (100, 1)])
def test_a_query_is_a_decode_of_a_shorter_sequence(window, sinks):
    """Without a window, query i is the decode of the sequence cut behind it; a window of one is the token's value."""
    rng = np.random.default_rng(2)
    t = tier(rng, [8])
    q = rng.standard_normal((8, 2, 64)).astype(np.float16)
    got = chunk.chunk_attention(q, [t], [0, 8], window, sinks)
    for i in range(8):
        if window == 1 and sinks == 0:
            want = np.stack([oatt.dequantised_kv([t], 0, g)[1][i] for g in range(2)])
        else:
            keep = np.flatnonzero(chunk.sees(i, 8, window, sinks))
            want = np.stack([oatt.attend(q[i, g].astype(np.float64), *(x[keep] for x in oatt.dequantised_kv([t], 0, g)))
                             for g in range(2)])
        assert np.allclose(got[i], want, rtol=0, atol=1e-12)


def test_a_chunk_longer_than_its_sequence():
    rng = np.random.default_rng(3)
    t = tier(rng, [2])
    q = rng.standard_normal((5, 2, 64)).astype(np.float16)
    got = chunk.chunk_attention(q, [t], [0, 5])
    assert not got[:3].any() and got[3:].any(-1).all()
