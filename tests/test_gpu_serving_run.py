"""The serving operators together, as a decode loop uses them: a prompt chunk is turned and appended
(kvq_rope_append), then every step turns the sequences' queries, appends their new tokens, attends
over the shared prompt and their own tokens (kvq_decode_attention_shared) and reads the new tokens
back (kvq_dequantize).  The step is captured once; positions, slots and lengths are read when it is
replayed.

Tolerances, derived before the first run, u = 2^-11 (half an ulp of fp16).  Read-back vectors are
what attention sees, rounded once: attention on them in float64 differs from the call's by the
call's own 4 u (2-norm of all outputs against the outputs', as in tests/test_gpu_shared.py) and the
read-back's roundings of keys (scores of unit variance: u) and values (u), added in squares below
4.3 u; the queries it is given are the turned ones as they were written, fp16, so they add nothing.
5 u are allowed.  An fp16 cache rounds the rotated vector once and the read-back the vector once,
each by at most u of the 2-norm (2^-25 a coordinate where it is subnormal); cos, sin and the
transforms, in float32, stay below 2^-18."""
import math

import numpy as np
import pytest

from oracle import rope as orope
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -11

FORMATS = {"fp16": ("fp16", "fp16", 0), "fp8_int4": ("fp8_e4m3", "int4_g32", 0), "cb4": ("codebook", "codebook", 4)}


@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 64)])
@pytest.mark.parametrize("name", list(FORMATS))
def test_decode_loop(name, layout, rot):
    torch, kvq = gu.torch_cuda(), gu.kvq_module()
    kf, vf, bits = FORMATS[name]
    hkv, hq, d, ps, batch, prompt, steps = 8, 32, 128, 16, 6, 2100, 5  # 2100 x 8 vectors: the large append
    rng = np.random.default_rng(rot)
    ks, vs = (np.where(rng.integers(0, 2, (hkv, d)) == 0, 1, -1).astype(np.int8) for _ in range(2))
    prompt_pages, total = -(-prompt // ps), -(-prompt // ps) + batch
    cache = kvq.PagedCache(d, hkv, total, kf, vf, bits, bits, ks, vs, ps)
    rope = kvq.Rope(rot, layout, base=500000.0)
    w = orope.frequencies(500000.0, rot)
    perm = rng.permutation(total).astype(np.int32)
    slot = lambda page, t: int(perm[page]) * ps + t % ps  # noqa: E731

    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    half = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
    # ---- the prompt, from one projection's output: strided views of q, k and v
    qkv = half(prompt, hq + 2 * hkv, d)
    x = dev(qkv)
    pos = np.arange(prompt, dtype=np.int32)
    slots = np.array([slot(t // ps, t) for t in range(prompt)], np.int32)
    kvq.kvq_rope_append(cache.struct, rope, dev(pos), x[:, hq:hq + hkv], x[:, hq + hkv:], dev(slots), q=x[:, :hq])
    torch.cuda.synchronize()
    got = x.cpu().numpy()
    assert np.array_equal(got[:, hq:], qkv[:, hq:])  # keys and values are only read
    want = orope.apply(qkv[:, :hq], pos, w, layout)
    assert np.all(np.abs(got[:, :hq] - want) <= U * np.abs(want) + 2.0 ** -18 * np.abs(want).max() + 2.0 ** -25)

    # ---- the decode loop
    prefix = kvq.TierView(cache, dev(perm[None, :prompt_pages]), dev(np.array([prompt], np.int32)))
    own_lens = dev(np.zeros(batch, np.int32))
    own = kvq.TierView(cache, dev(perm[prompt_pages:, None]), own_lens)
    offsets = [0, batch]
    step = torch.empty(batch, hq + 2 * hkv, d, dtype=torch.float16, device="cuda")
    q, k, v = step[:, :hq], step[:, hq:hq + hkv], step[:, hq + hkv:]
    q_out = torch.empty(batch, hq, d, dtype=torch.float16, device="cuda")
    out, kb, vb = torch.empty_like(q_out), torch.empty(batch, hkv, d, dtype=torch.float16, device="cuda"), None
    vb = torch.empty_like(kb)
    positions, new_slots = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(kvq.kvq_decode_shared_workspace_size([prefix], offsets, [own], batch, hq), dtype=torch.uint8,
                     device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        kvq.kvq_rope_append(cache.struct, rope, positions, k, v, new_slots, q=q, q_out=q_out)
        kvq.kvq_decode_attention_shared([prefix], offsets, [own], q_out, out, ws, status)
        kvq.kvq_dequantize(cache.struct, new_slots, kb, vb)

    graph = None
    keys, values = [], []  # per step [batch, hkv, d], as read back
    everything = dev(slots)
    pk, pv = (torch.empty(prompt, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    kvq.kvq_dequantize(cache.struct, everything, pk, pv)
    torch.cuda.synchronize()
    pk, pv = pk.cpu().numpy().astype(np.float64), pv.cpu().numpy().astype(np.float64)
    if name == "fp16":
        turned = orope.apply(qkv[:, hq:hq + hkv], pos, w, layout)
        size = np.linalg.norm(turned, axis=-1)
        assert np.all(np.linalg.norm(pk - turned, axis=-1) <= (2 * U + 2.0 ** -18) * size + 2.0 ** -25 * 2 * math.sqrt(d))
    for i in range(steps):
        new = half(batch, hq + 2 * hkv, d)
        step.copy_(dev(new))
        positions.copy_(dev(np.full(batch, prompt + i, np.int32)))
        new_slots.copy_(dev(np.array([slot(prompt_pages + b, i) for b in range(batch)], np.int32)))
        own_lens.fill_(i + 1)
        if i < 2:
            run()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run()
            graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        keys.append(kb.cpu().numpy().astype(np.float64))
        values.append(vb.cpu().numpy().astype(np.float64))
        if name == "fp16":
            turned = orope.apply(new[:, hq:hq + hkv], np.full(batch, prompt + i), w, layout)
            size = np.linalg.norm(turned, axis=-1)
            assert np.all(np.linalg.norm(keys[-1] - turned, axis=-1)
                          <= (2 * U + 2.0 ** -18) * size + 2.0 ** -25 * 2 * math.sqrt(d))
        qt = q_out.cpu().numpy().astype(np.float64)
        got = out.cpu().numpy().astype(np.float64)
        off = total_size = 0.0
        for b in range(batch):
            for h in range(hq):
                kk = np.concatenate([pk[:, h // 4], np.stack([s[b, h // 4] for s in keys])])
                vv = np.concatenate([pv[:, h // 4], np.stack([s[b, h // 4] for s in values])])
                s = kk @ qt[b, h] / math.sqrt(d)
                p = np.exp(s - s.max())
                want = (p / p.sum()) @ vv
                off += float(np.sum((got[b, h] - want) ** 2))
                total_size += float(np.sum(want ** 2))
        assert math.sqrt(off / total_size) <= 5 * U, math.sqrt(off / total_size)
