"""What the cache's attention over chunks of tokens and over windows is measured on.

Two operators on the quantised, paged KV cache:

* ``chunk``: attention of the newest tokens of every sequence (a prompt's chunk, drafted tokens
  to be checked, a step's single token) over all that the sequence has cached, themselves
  included, each token seeing what stands at or before it; with a sliding window and a few first
  tokens that stay visible (sinks), or without;
* ``window``: the decode step of layers with such a window: one query per sequence over the
  sinks and the window.

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the
framework's calls.  ``exact`` is their definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16  # tokens per page
# formats: (key format, value format, key bits, value bits)
FORMATS = {
    "fp16": ("fp16", "fp16", 0, 0),
    "fp8_int4": ("fp8_e4m3", "int4_g32", 0, 0),
    "cb4": ("codebook", "codebook", 4, 4),
    "cb32": ("codebook", "codebook", 3, 2),
}


# --------------------------------------------------------------------------- cases
# tokens: the longest chunk (1: a decode step); context: the most tokens cached before it;
# recent: the newest tokens that are kept in an fp16 tier of their own; window 0: no window
def listed():
    return [
        # drafted tokens of a few sequences, to be checked in one pass
        {"name": "chunk_draft", "op": "chunk", "batch": 4, "tokens": 5, "context": 2000, "hq": 32, "hkv": 8, "dim": 128,
         "format": "fp8_int4", "recent": 0, "window": 0, "sinks": 0, "ragged": False},
        # a whole prompt, one query head per kv head
        {"name": "chunk_prompt", "op": "chunk", "batch": 1, "tokens": 4096, "context": 0, "hq": 32, "hkv": 32, "dim": 128,
         "format": "cb4", "recent": 0, "window": 0, "sinks": 0, "ragged": False},
        # a chunk of a long prompt with grouped heads
        {"name": "chunk_long", "op": "chunk", "batch": 1, "tokens": 4096, "context": 28672, "hq": 32, "hkv": 8, "dim": 128,
         "format": "fp8_int4", "recent": 0, "window": 0, "sinks": 0, "ragged": False},
        # a scheduler's mixed step: chunks and single tokens of sequences of all lengths
        {"name": "chunk_ragged", "op": "chunk", "batch": 16, "tokens": 333, "context": 8000, "hq": 32, "hkv": 8, "dim": 128,
         "format": "cb32", "recent": 0, "window": 0, "sinks": 0, "ragged": True},
        # wide heads
        {"name": "chunk_wide", "op": "chunk", "batch": 2, "tokens": 512, "context": 16384, "hq": 16, "hkv": 16, "dim": 256,
         "format": "cb4", "recent": 0, "window": 0, "sinks": 0, "ragged": False},
        # narrow heads, an odd chunk
        {"name": "chunk_narrow", "op": "chunk", "batch": 3, "tokens": 777, "context": 5001, "hq": 16, "hkv": 4, "dim": 64,
         "format": "fp16", "recent": 0, "window": 0, "sinks": 0, "ragged": False},
        # older tokens quantised, the newest in an fp16 tier
        {"name": "chunk_tiers", "op": "chunk", "batch": 8, "tokens": 64, "context": 8192, "hq": 32, "hkv": 8, "dim": 128,
         "format": "fp8_int4", "recent": 256, "window": 0, "sinks": 0, "ragged": True},
        # the same layer's chunk under a sliding window with sinks
        {"name": "chunk_window", "op": "chunk", "batch": 2, "tokens": 2048, "context": 30000, "hq": 32, "hkv": 8, "dim": 128,
         "format": "fp16", "recent": 0, "window": 4096, "sinks": 4, "ragged": False},
        # a decode step of one sequence, far behind its first tokens
        {"name": "window_single", "op": "window", "batch": 1, "tokens": 1, "context": 16000, "hq": 8, "hkv": 8, "dim": 128,
         "format": "cb4", "recent": 0, "window": 512, "sinks": 4, "ragged": False},
        # a batch of grouped heads with a long window
        {"name": "window_batch", "op": "window", "batch": 64, "tokens": 1, "context": 20000, "hq": 32, "hkv": 8, "dim": 128,
         "format": "fp8_int4", "recent": 0, "window": 4096, "sinks": 4, "ragged": True},
        # one query head per kv head, packed codes
        {"name": "window_codes", "op": "window", "batch": 16, "tokens": 1, "context": 8191, "hq": 32, "hkv": 32, "dim": 128,
         "format": "cb4", "recent": 0, "window": 2048, "sinks": 16, "ragged": False},
        # wide heads, odd sizes
        {"name": "window_wide", "op": "window", "batch": 32, "tokens": 1, "context": 6001, "hq": 16, "hkv": 8, "dim": 256,
         "format": "cb32", "recent": 0, "window": 1021, "sinks": 1, "ragged": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "window"])
    dim = rng.choice([64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    hq = hkv * rng.choice([1, 2, 4, 8] if hkv <= 8 else [1, 2])
    windowed = op == "window" or rng.random() < 0.4
    window, sinks = (_log_int(rng, 16, 8192), rng.choice([0, 1, 4, 4, 16, 100])) if windowed else (0, 0)
    batch = _log_int(rng, 1, 64)
    tokens = 1 if op == "window" else _log_int(rng, 1, 4096 if batch == 1 else max(2, 4096 // batch))
    # no more work than the largest listed case, and vectors and scores of the plain form that fit the card
    most = min(32 * 4096 * 30720 * 128 // (batch * tokens * hq * dim), 4 * 10 ** 9 // (batch * tokens * hq),
               10 ** 9 // (batch * hkv * dim), 65536) - tokens
    context = _log_int(rng, 1, max(2, most)) - 1
    return {"op": op, "batch": batch, "tokens": tokens, "context": context, "hq": hq, "hkv": hkv, "dim": dim,
            "format": rng.choice(sorted(FORMATS)), "recent": rng.choice([0, 0, 0, 64, 500]), "window": window,
            "sinks": sinks, "ragged": rng.random() < 0.5}


# --------------------------------------------------------------------------- the cache's formats
_TABLES = {}


def _table(bits):
    """Lloyd-Max centroids of N(0, 1) with 2^bits levels and the midpoints between them."""
    if bits not in _TABLES:
        cdf = np.vectorize(lambda x: 0.5 * (1.0 + math.erf(x / math.sqrt(2.0))))
        pdf = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)  # noqa: E731
        c = np.linspace(-2.5, 2.5, 2 ** bits)
        for _ in range(4000):
            edge = np.concatenate([[-8.0], 0.5 * (c[1:] + c[:-1]), [8.0]])
            new = (pdf(edge[:-1]) - pdf(edge[1:])) / (cdf(edge[1:]) - cdf(edge[:-1]))
            done = np.abs(new - c).max() < 1e-13
            c = new
            if done:
                break
        c32 = c.astype(np.float32)
        b32 = (0.5 * (c32[1:].astype(np.float64) + c32[:-1].astype(np.float64))).astype(np.float32)
        _TABLES[bits] = c32, b32
    return _TABLES[bits]


_HADAMARDS = {}


def _hadamard(d):
    if d not in _HADAMARDS:
        i = np.arange(d)
        ones = sum((i[:, None] & i) >> bit & 1 for bit in range(d.bit_length()))  # common bits of row and column
        _HADAMARDS[d] = torch.from_numpy(1.0 - 2.0 * (ones % 2)).float().cuda()
    return _HADAMARDS[d]


def _encode(x, fmt, bits):
    """Rotated vectors [..., d] -> (rows uint8 [..., row bytes], side data or None)."""
    d = x.shape[-1]
    if fmt == "fp16":
        return x.half().view(torch.uint8), None
    if fmt == "fp8_e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), None
    if fmt == "int4_g32":
        g = x.unflatten(-1, (d // 32, 32))
        scale = (g.abs().amax(-1) / 7.0).half()
        q = torch.where(scale[..., None] > 0, (g / scale[..., None].float()).round().clamp(-7, 7), torch.zeros_like(g))
        q = (q + 8).to(torch.uint8).flatten(-2)
        return q[..., 0::2] | (q[..., 1::2] << 4), scale
    norm = x.square().sum(-1, keepdim=True).sqrt()
    u = torch.where(norm > 0, x / norm * math.sqrt(d), torch.zeros_like(x))
    bounds = torch.from_numpy(_table(bits)[1]).cuda()
    codes = torch.bucketize(u, bounds).to(torch.uint8)  # the number of boundaries below u
    shifts = torch.arange(bits, device="cuda", dtype=torch.uint8)
    stream = ((codes[..., None] >> shifts) & 1).flatten(-2).unflatten(-1, (d * bits // 8, 8))
    weight = (2 ** torch.arange(8, device="cuda")).to(torch.uint8)
    return (stream * weight).sum(-1, dtype=torch.uint8), norm[..., 0].half()


def _decode(rows, aux, d, fmt, bits):
    """Stored rows -> the rotated vectors that they stand for."""
    if fmt == "fp16":
        return rows.view(torch.float16).float()
    if fmt == "fp8_e4m3":
        return rows.view(torch.float8_e4m3fn).float()
    if fmt == "int4_g32":
        q = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float() - 8.0
        return (q.unflatten(-1, (d // 32, 32)) * aux[..., None].float()).flatten(-2)
    j = torch.arange(d, device="cuda") * bits
    pad = torch.nn.functional.pad(rows, (0, 1)).to(torch.int16)
    word = pad[..., j // 8] | (pad[..., j // 8 + 1] << 8)
    codes = (word >> (j % 8).to(torch.int16)) & (2 ** bits - 1)
    return torch.from_numpy(_table(bits)[0]).cuda()[codes.long()] * aux[..., None].float() / math.sqrt(d)


def _outliers(gen, heads, d):
    pairs = torch.rand((heads, d), device="cuda", generator=gen) < 0.01
    return torch.where(pairs, 30.0, 1.0)


def _signs(gen, heads, d):
    return (torch.randint(0, 2, (heads, d), device="cuda", generator=gen) * 2 - 1).to(torch.int8)


def _pool(gen, num_pages, hkv, d, fmt, signs, large):
    """A filled cache: K and V rows and side data [pages, kv heads, page, ...], every slot holding a token like
    a layer's keys or values: normal, some (head, channel) pairs far larger."""
    pool = {}
    for i, side in enumerate("kv"):
        rows, aux = [], []
        for part in torch.arange(num_pages, device="cuda").split(4096):  # (the 32-bit vectors of a long cache are large)
            x = (torch.randn((len(part) * PAGE, hkv, d), device="cuda", generator=gen) * large[i]).half().float()
            r, a = _encode((x * signs[i].float()) @ _hadamard(d) / math.sqrt(d), fmt[i], fmt[2 + i])
            rows.append(r.unflatten(0, (len(part), PAGE)).transpose(1, 2).contiguous())
            aux.append(None if a is None else a.unflatten(0, (len(part), PAGE)).transpose(1, 2).contiguous())
        pool[side + "_rows"] = torch.cat(rows)
        pool[side + "_aux"] = None if aux[0] is None else torch.cat(aux)
    return pool


def _handle(tier, fmt, num_pages, hkv, d, signs):
    """The framework's cache object over a tier's pool."""
    import quantized_decode_attention_rht_gb300 as kvq
    cache = kvq.PagedCache(d, hkv, num_pages, fmt[0], fmt[1], fmt[2], fmt[3], signs[0], signs[1], PAGE)
    for name in ("k_rows", "v_rows", "k_aux", "v_aux"):
        if tier[name] is not None:
            own_buffer = getattr(cache, name)
            own_buffer.copy_(tier[name].view(own_buffer.shape))
            tier[name] = own_buffer.view(tier[name].shape)
    return cache


# --------------------------------------------------------------------------- states
def _lengths(case, seed):
    """Per sequence (host): the chunk's tokens, the case's own, and all cached tokens, the chunk's among them."""
    b, most = case["batch"], case["tokens"]
    if not case["ragged"]:
        return [most] * b, [case["context"] + most] * b
    draws = torch.rand(b, generator=torch.Generator().manual_seed(most)).tolist()
    tokens = [max(1, round(math.exp(x * math.log(most)))) for x in draws]
    context = [round(x * case["context"]) for x in torch.rand(b, generator=torch.Generator().manual_seed(seed)).tolist()]
    tokens[0], context[0] = most, case["context"]
    return tokens, [t + c for t, c in zip(tokens, context)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["dim"]
    tokens, lens = _lengths(case, int(seed))
    signs = [_signs(gen, hkv, d), _signs(gen, hkv, d)]
    large = [_outliers(gen, hkv, d), _outliers(gen, hkv, d)]
    s = {"case": case, "signs": signs, "tiers": [], "tokens": tokens, "lens": lens}
    # oldest tokens first: the quantised tier, then the fp16 tier of the newest ones
    recent = [min(case["recent"], n) for n in lens]
    kept = [(FORMATS[case["format"]], [n - r for n, r in zip(lens, recent)])]
    if case["recent"]:
        kept.append((FORMATS["fp16"], recent))
    for fmt, held in kept:
        pages = [-(-n // PAGE) for n in held]
        total, width = max(1, sum(pages)), max(1, max(pages))
        tier = _pool(gen, total, hkv, d, fmt, signs, large)
        order = torch.randperm(total, device="cuda", generator=gen).to(torch.int32)
        column = torch.arange(width, device="cuda")[None, :]
        first = torch.tensor(np.cumsum([0] + pages[:-1]), device="cuda")[:, None]
        there = column < torch.tensor(pages, device="cuda")[:, None]
        tier["table"] = torch.where(there, order[(first + column).clamp(max=total - 1)], 0).to(torch.int32).contiguous()
        tier["lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")
        tier["fmt"] = fmt
        s["tiers"].append(tier)
        if own:
            import quantized_decode_attention_rht_gb300 as kvq
            tier["cache"] = _handle(tier, fmt, total, hkv, d, signs)
            s.setdefault("views", []).append(kvq.TierView(tier["cache"], tier["table"], tier["lens"]))
    n = sum(tokens)
    s["offsets"] = torch.tensor([0] + list(np.cumsum(tokens)), dtype=torch.int32, device="cuda")
    s["all_lens"] = torch.tensor(lens, device="cuda")
    s["q"] = torch.randn((n, hq, d), device="cuda", generator=gen).half()
    if own:
        s["out"] = torch.empty((n, hq, d), dtype=torch.float16, device="cuda")
        if case["op"] == "chunk":
            need = kvq.kvq_chunk_workspace_size(s["views"], b, n, hq, window=case["window"], sinks=case["sinks"])
        else:
            need = kvq.kvq_decode_window_workspace_size(s["views"], b, hq, case["window"], case["sinks"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass
def _stored(tier, side, signs, positions):
    """A tier's tokens at `positions` [b, n] of its sequences, as the vectors that they stand for: [b, kv heads, n, d]."""
    i = 0 if side == "k" else 1
    fmt, bits = tier["fmt"][i], tier["fmt"][2 + i]
    page = tier["table"].gather(1, positions // PAGE).long()
    rows = tier[side + "_rows"][page, :, positions % PAGE]
    aux = tier[side + "_aux"]
    aux = None if aux is None else aux[page, :, positions % PAGE]
    d = signs[i].shape[-1]
    return ((_decode(rows, aux, d, fmt, bits) @ _hadamard(d)) / math.sqrt(d) * signs[i].float()).transpose(1, 2)


def run(s):
    c = s["case"]
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        if c["op"] == "chunk":
            kvq.kvq_chunk_attention(s["views"], s["offsets"], s["q"], s["out"], s["workspace"], window=c["window"],
                                    sinks=c["sinks"])
        else:
            kvq.kvq_decode_attention_window(s["views"], s["q"], s["out"], s["workspace"], c["window"], c["sinks"])
        return s["out"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["dim"]
    g, most, longest = hq // hkv, max(s["tokens"]), max(s["lens"])
    lens, tokens = s["all_lens"][:, None], (s["offsets"][1:] - s["offsets"][:-1]).long()[:, None]
    # the queries, side by side per kv head, and where they stand
    i = torch.arange(most, device="cuda")[None, :]
    at = lens - tokens + i  # [b, most]
    row = (s["offsets"][:-1, None] + torch.minimum(i, tokens - 1)).long()
    q = s["q"][row].float().view(b, most, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, most * g, d) / math.sqrt(d)
    # the positions that any of them may see: from the first one's window on, and the sinks before it
    if c["window"]:
        begin = (at[:, :1] - c["window"] + 1).clamp(min=0)
        width = min(longest, most + c["window"] - 1)
        t = begin + torch.arange(width, device="cuda")[None, :]
        first = torch.arange(min(c["sinks"], longest), device="cuda")[None, :].expand(b, -1)
        t = torch.cat([torch.where(first < begin, first, longest), t], 1)
    else:
        t = torch.arange(longest, device="cuda")[None, :].expand(b, -1)
    k = v = None
    base = torch.zeros_like(lens)
    for tier in s["tiers"]:
        held = tier["lens"].long()[:, None]
        where = (t - base).clamp(min=0)
        where = torch.minimum(where, (held - 1).clamp(min=0))
        tk, tv = _stored(tier, "k", s["signs"], where), _stored(tier, "v", s["signs"], where)
        later = ((t >= base) & (t < base + held))[:, None, :, None]
        k, v = (tk, tv) if k is None else (torch.where(later, tk, k), torch.where(later, tv, v))
        base = base + held
    seen = (t[:, None, :] <= at[:, :, None]) & (t < lens)[:, None, :]
    if c["window"]:
        seen &= (t[:, None, :] > at[:, :, None] - c["window"]) | (t < c["sinks"])[:, None, :]
    p = q @ k.transpose(-1, -2)
    p = p.view(b, hkv, most, g, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf).view(p.shape)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    out = p @ v
    out = (out / torch.where(total > 0, total, torch.ones_like(total))).view(b, hkv, most, g, d)
    return out.permute(0, 2, 1, 3, 4).reshape(b, most, hq, d)[i < tokens].half()


# --------------------------------------------------------------------------- work
def _row_bytes(name, bits, d):
    return {"fp16": 2 * d, "fp8_e4m3": d, "int4_g32": d // 2 + d // 16, "codebook": d * bits // 8 + 2}[name]


def _token_bytes(name, d):
    """Bytes of one cached token of one kv head."""
    fmt = FORMATS[name]
    return _row_bytes(fmt[0], fmt[2], d) + _row_bytes(fmt[1], fmt[3], d)


def work(case):
    d, hq, hkv, window, sinks = case["dim"], case["hq"], case["hkv"], case["window"], case["sinks"]
    tokens, lens = _lengths(case, 0)  # of one seed: the lengths vary a little with it
    pairs = cached = 0
    for t, n in zip(tokens, lens):
        p = np.arange(n - t, n, dtype=np.float64)
        begin = np.maximum(p - window + 1, 0) if window else 0 * p
        pairs += float((p + 1 - begin + np.minimum(begin, sinks)).sum())
        seen = n - begin[0] + min(begin[0], sinks)  # tokens that some query sees
        new = min(case["recent"], n, seen)
        cached += hkv * (new * _token_bytes("fp16", d) + (seen - new) * _token_bytes(case["format"], d))
    return {"bytes": float(cached) + 4.0 * sum(tokens) * hq * d, "flops": 4.0 * pairs * hq * d}


# --------------------------------------------------------------------------- 64 bits
def _exact_butterflies(x):
    """Walsh-Hadamard transform of the last axis / sqrt(d), in 64 bits."""
    d = x.shape[-1]
    y, step = x.double(), 1
    while step < d:
        y = y.reshape(*x.shape[:-1], d // (2 * step), 2, step)
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        step *= 2
    return y / math.sqrt(d)


def _exact_stored(tier, side, signs, sequence, count):
    """The first `count` tokens of a sequence in a tier, in 64 bits: [count, kv heads, d], the bits of the
    rows taken apart one field at a time."""
    i = 0 if side == "k" else 1
    fmt, bits, d = tier["fmt"][i], tier["fmt"][2 + i], signs[i].shape[-1]
    t = torch.arange(count, device="cuda")
    page, off = tier["table"][sequence].long()[t // PAGE], t % PAGE
    rows = tier[side + "_rows"].transpose(1, 2)[page, off]
    aux = tier[side + "_aux"]
    aux = None if aux is None else aux.transpose(1, 2)[page, off].double()
    if fmt == "fp16":
        x = rows.contiguous().view(torch.float16).double()
    elif fmt == "fp8_e4m3":
        r = rows.long()
        e, m, sign = (r >> 3) & 15, (r & 7).double(), 1.0 - 2.0 * (r >> 7).double()
        x = sign * torch.where(e > 0, (8.0 + m) * 2.0 ** (e.double() - 10.0), m * 2.0 ** -9)
    elif fmt == "int4_g32":
        x = torch.empty(*rows.shape[:-1], d, dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = (rows % 16).double() - 8.0, torch.div(rows, 16, rounding_mode="floor").double() - 8.0
        x = x * aux.repeat_interleave(32, -1)
    else:
        cent = torch.from_numpy(_table(bits)[0]).cuda().double()
        x = torch.empty(*rows.shape[:-1], d, dtype=torch.float64, device="cuda")
        for j in range(d):
            byte, shift = (j * bits) // 8, (j * bits) % 8
            field = rows[..., byte].long()
            if shift + bits > 8:
                field = field + 256 * rows[..., byte + 1].long()
            x[..., j] = cent[(field >> shift) % (2 ** bits)]
        x = x * aux[..., None] / math.sqrt(d)
    return _exact_butterflies(x) * signs[i].double()


def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]
    out = torch.empty((sum(s["tokens"]), hq, d), dtype=torch.float64, device="cuda")
    done = 0
    for j, (count, length) in enumerate(zip(s["tokens"], s["lens"])):
        k, v = (torch.cat([_exact_stored(tier, x, s["signs"], j, int(tier["lens"][j])) for tier in s["tiers"]])
                .transpose(0, 1) for x in "kv")
        t = torch.arange(length, device="cuda")
        rows = max(1, 10 ** 9 // (hq * length))  # tokens at a time, their scores being large
        for first in range(0, count, rows):
            last = min(count, first + rows)
            p = length - count + torch.arange(first, last, device="cuda")[:, None]
            hidden = t > p
            if case["window"]:
                hidden |= (p - t >= case["window"]) & (t >= case["sinks"])
            q = s["q"][done + first:done + last].double().reshape(last - first, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            w = torch.matmul(q, k[:, None].transpose(2, 3)) / math.sqrt(d)
            w[:, :, hidden] = -math.inf
            y = torch.matmul(torch.softmax(w, -1), v[:, None])  # (every query sees itself at least)
            out[done + first:done + last] = y.permute(2, 0, 1, 3).reshape(last - first, hq, d)
        done += count
    return out
