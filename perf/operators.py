"""What the cache's serving operators are measured on.

Four operators around the quantised KV cache:

* ``rope``: rotary positions of queries and keys (and the transpose, its gradient);
* ``append``: rotary positions, rotation, encoding and storing of new tokens in one call,
  then the tokens read back as the cache holds them;
* ``read``: cached tokens read back as fp16 vectors;
* ``shared``: decode attention for groups of sequences that share a cached prefix, each with
  a cached continuation of its own.

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
def listed():
    return [
        # one decode step of 64 sequences at long positions, q and k views of one fused projection
        {"name": "rope_step", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "by_parts", "start": 65536, "grad": False},
        # a prompt chunk: wide heads, half of each rotated, neighbouring pairs
        {"name": "rope_chunk", "op": "rope", "tokens": 16384, "hq": 16, "hkv": 16, "dim": 256, "rot": 128,
         "layout": "interleaved", "scaling": "linear", "start": 131072, "grad": False},
        # the gradient of a training sequence of odd length
        {"name": "rope_gradient", "op": "rope", "tokens": 4097, "hq": 32, "hkv": 32, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "start": 0, "grad": True},
        # the new token of every sequence of a decode step
        {"name": "append_step", "op": "append", "tokens": 32, "hq": 32, "hkv": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "by_parts", "start": 32768, "format": "fp8_int4"},
        # a prompt chunk after a long cached context
        {"name": "append_chunk", "op": "append", "tokens": 16384, "hq": 16, "hkv": 16, "dim": 256, "rot": 256,
         "layout": "half", "scaling": "base", "start": 131072, "format": "cb4"},
        # a few tokens of scattered pages
        {"name": "read_some", "op": "read", "tokens": 333, "hkv": 8, "dim": 128, "format": "cb32"},
        # a whole context of one layer
        {"name": "read_context", "op": "read", "tokens": 65536, "hkv": 8, "dim": 128, "format": "fp8_int4"},
        # two sequences on a short prompt
        {"name": "shared_pair", "op": "shared", "batch": 2, "groups": 1, "hq": 8, "hkv": 8, "dim": 128,
         "prefix": 1000, "suffix": 24, "format": "cb4"},
        # samples of one prompt, one query head per kv head
        {"name": "shared_samples", "op": "shared", "batch": 8, "groups": 1, "hq": 32, "hkv": 32, "dim": 128,
         "prefix": 8192, "suffix": 256, "format": "cb4"},
        # grouped heads on a long context
        {"name": "shared_context", "op": "shared", "batch": 32, "groups": 1, "hq": 32, "hkv": 8, "dim": 128,
         "prefix": 32768, "suffix": 512, "format": "fp8_int4"},
        # several prompts of different lengths, shared by different numbers of sequences
        {"name": "shared_ragged", "op": "shared", "batch": 64, "groups": 5, "hq": 32, "hkv": 8, "dim": 128,
         "prefix": 20011, "suffix": 333, "format": "cb32"},
        # a full batch on one system prompt
        {"name": "shared_batch", "op": "shared", "batch": 256, "groups": 1, "hq": 64, "hkv": 8, "dim": 128,
         "prefix": 16384, "suffix": 128, "format": "fp8_int4"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "shared", "shared"])
    if op == "shared":
        hkv = rng.choice([4, 8, 16, 32])
        hq = hkv * rng.choice([1, 2, 4, 8] if hkv <= 8 else [1, 2])
        batch = _log_int(rng, 2, 256)
        # no more work than the largest listed case
        most = 256 * 64 * 16384 // (batch * hq)
        prefix = _log_int(rng, 100, max(200, min(65536, most)))
        return {"op": op, "batch": batch, "groups": rng.choice([1, 1, 2, 3, 7]), "hq": hq, "hkv": hkv, "dim": 128,
                "prefix": prefix, "suffix": _log_int(rng, 1, 512), "format": rng.choice(sorted(FORMATS))}
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    tokens = _log_int(rng, 1, 65536 * 8 * 128 // (hkv * dim) // (1 if op == "read" else 4))
    if op == "read":
        return {"op": op, "tokens": tokens, "hkv": hkv, "dim": dim, "format": rng.choice(sorted(FORMATS))}
    hq = hkv * rng.choice([1, 2, 4])
    rot = rng.choice([dim, dim, dim, dim // 2, dim // 4])
    case = {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "rot": rot,
            "layout": rng.choice(["half", "interleaved"]),
            "scaling": rng.choice(["none", "linear", "base", "by_parts"]), "start": _log_int(rng, 1, 1 << 20) - 1}
    if op == "rope":
        case["grad"] = rng.random() < 0.3
    else:
        case["format"] = rng.choice(sorted(FORMATS))
    return case


# --------------------------------------------------------------------------- rotary frequencies
ROPE_BASE = 500000.0
# kind -> (factor, original context, low turns, high turns, attention scale)
SCALINGS = {"none": (1.0, 0.0, 0.0, 0.0, 1.0), "linear": (4.0, 0.0, 0.0, 0.0, 1.0), "base": (8.0, 0.0, 0.0, 0.0, 1.0),
            "by_parts": (8.0, 8192.0, 1.0, 32.0, 0.1 * math.log(8.0) + 1.0)}


def _frequencies(rot, kind):
    """Radians per token of each pair, in 64 bits, and the factor of cos and sin."""
    factor, context, low, high, scale = SCALINGS[kind]
    base = ROPE_BASE * factor ** (rot / (rot - 2.0)) if kind == "base" and rot > 2 else ROPE_BASE
    w = base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    if kind == "linear":
        w = w / factor
    elif kind == "by_parts":
        keep = np.clip((context * w / (2.0 * math.pi) - low) / (high - low), 0.0, 1.0)
        w = w * (keep + (1.0 - keep) / factor)
    return w, scale


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


def _hadamard(d, dtype):
    if (d, dtype) not in _HADAMARDS:
        i = np.arange(d)
        ones = sum((i[:, None] & i) >> bit & 1 for bit in range(d.bit_length()))  # common bits of row and column
        _HADAMARDS[d, dtype] = torch.from_numpy(1.0 - 2.0 * (ones % 2)).to(dtype).cuda()
    return _HADAMARDS[d, dtype]


def _rotate(x, signs, dtype=torch.float32):
    """x [..., heads, d] -> H (s x) / sqrt(d)."""
    d = x.shape[-1]
    return (x.to(dtype) * signs.to(dtype)) @ _hadamard(d, dtype) / math.sqrt(d)


def _unrotate(x, signs, dtype=torch.float32):
    d = x.shape[-1]
    return (x.to(dtype) @ _hadamard(d, dtype)) / math.sqrt(d) * signs.to(dtype)


def _encode(x, fmt, bits):
    """Rotated vectors [..., d] -> (rows uint8 [..., row bytes], side data or None)."""
    d = x.shape[-1]
    if fmt == "fp16":
        return x.half().view(torch.uint8), None
    if fmt == "fp8_e4m3":
        return x.float().clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), None
    if fmt == "int4_g32":
        g = x.unflatten(-1, (d // 32, 32)).float()
        scale = (g.abs().amax(-1) / 7.0).half()
        q = torch.where(scale[..., None] > 0, (g / scale[..., None].float()).round().clamp(-7, 7), torch.zeros_like(g))
        q = (q + 8).to(torch.uint8).flatten(-2)
        return q[..., 0::2] | (q[..., 1::2] << 4), scale
    norm = x.square().sum(-1, keepdim=True).sqrt()
    u = torch.where(norm > 0, x / norm * math.sqrt(d), torch.zeros_like(x)).float()
    bounds = torch.from_numpy(_table(bits)[1]).cuda()
    codes = torch.bucketize(u, bounds).to(torch.uint8)  # the number of boundaries below u
    shifts = torch.arange(bits, device="cuda", dtype=torch.uint8)
    stream = ((codes[..., None] >> shifts) & 1).flatten(-2).unflatten(-1, (d * bits // 8, 8))
    weight = (2 ** torch.arange(8, device="cuda")).to(torch.uint8)
    return (stream * weight).sum(-1, dtype=torch.uint8), norm[..., 0].half()


def _decode(rows, aux, d, fmt, bits, dtype=torch.float32):
    """Stored rows -> the rotated vectors that they stand for."""
    if fmt == "fp16":
        return rows.view(torch.float16).to(dtype)
    if fmt == "fp8_e4m3":
        return rows.view(torch.float8_e4m3fn).to(dtype)
    if fmt == "int4_g32":
        q = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).to(dtype) - 8.0
        return (q.unflatten(-1, (d // 32, 32)) * aux[..., None].to(dtype)).flatten(-2)
    j = torch.arange(d, device="cuda") * bits
    pad = torch.nn.functional.pad(rows, (0, 1)).to(torch.int16)
    word = pad[..., j // 8] | (pad[..., j // 8 + 1] << 8)
    codes = (word >> (j % 8).to(torch.int16)) & (2 ** bits - 1)
    return torch.from_numpy(_table(bits)[0]).cuda().to(dtype)[codes.long()] * aux[..., None].to(dtype) / math.sqrt(d)


def _draw_vectors(gen, n, heads, d, outliers):
    """fp16 vectors like a layer's keys or values: normal, some (head, channel) pairs far larger."""
    x = torch.randn((n, heads, d), device="cuda", generator=gen)
    return (x * outliers).half()


def _outliers(gen, heads, d):
    pairs = torch.rand((heads, d), device="cuda", generator=gen) < 0.01
    return torch.where(pairs, 30.0, 1.0)


def _signs(gen, heads, d):
    return (torch.randint(0, 2, (heads, d), device="cuda", generator=gen) * 2 - 1).to(torch.int8)


def _pool(gen, num_pages, hkv, d, fmt, ks, vs):
    """A filled cache: K and V rows and side data [pages, kv heads, page, ...], every slot holding a token."""
    pool = {}
    for side, name, bits, signs in (("k", fmt[0], fmt[2], ks), ("v", fmt[1], fmt[3], vs)):
        x = _draw_vectors(gen, num_pages * PAGE, hkv, d, _outliers(gen, hkv, d))
        rows, aux = _encode(_rotate(x, signs), name, bits)
        pool[side + "_rows"] = rows.unflatten(0, (num_pages, PAGE)).transpose(1, 2).contiguous()
        pool[side + "_aux"] = None if aux is None else aux.unflatten(0, (num_pages, PAGE)).transpose(1, 2).contiguous()
    return pool


def _empty_pool(num_pages, hkv, d, fmt):
    pool = {}
    for side, name, bits in (("k", fmt[0], fmt[2]), ("v", fmt[1], fmt[3])):
        rows, aux = _encode(torch.zeros((num_pages, hkv, PAGE, d), device="cuda"), name, bits)
        pool[side + "_rows"], pool[side + "_aux"] = rows, aux
    return pool


def _handle(s, fmt, num_pages, hkv, d):
    """The framework's cache object over the state's pool."""
    import quantized_decode_attention_rht_gb300 as kvq
    cache = kvq.PagedCache(d, hkv, num_pages, fmt[0], fmt[1], fmt[2], fmt[3], s["ks"], s["vs"], PAGE)
    for name in ("k_rows", "v_rows", "k_aux", "v_aux"):
        if s[name] is not None:
            own_buffer = getattr(cache, name)
            own_buffer.copy_(s[name].view(own_buffer.shape))
            s[name] = own_buffer.view(s[name].shape)
    return cache


# --------------------------------------------------------------------------- states
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"rope": _prepare_rope, "append": _prepare_append, "read": _prepare_read,
            "shared": _prepare_shared}[case["op"]](case, gen)


def _prepare_tokens(case, gen):
    """New tokens of a layer: q, k and v as views of one projection's output, and their positions."""
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["dim"]
    x = torch.randn((t, hq + 2 * hkv, d), device="cuda", generator=gen)
    x[:, hq:] *= _outliers(gen, 2 * hkv, d)
    x = x.half()
    s = {"case": case, "q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:]}
    if t <= 256:  # a decode step: every sequence at a place of its own
        s["positions"] = (case["start"] + torch.randint(0, 4096, (t,), device="cuda", generator=gen)).to(torch.int32)
    else:  # a chunk
        s["positions"] = torch.arange(case["start"], case["start"] + t, device="cuda", dtype=torch.int32)
    w, scale = _frequencies(case["rot"], case["scaling"])
    s["w"], s["scale"] = torch.from_numpy(w).cuda(), scale
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        factor, context, low, high, scale = SCALINGS[case["scaling"]]
        s["rope"] = kvq.Rope(case["rot"], case["layout"], base=ROPE_BASE, scaling=case["scaling"], factor=factor,
                             original_context=context, low_turns=low, high_turns=high, scale=scale)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.float16, device="cuda")
    return s


def _prepare_rope(case, gen):
    s = _prepare_tokens(case, gen)
    if own:
        s["k_out"] = torch.empty((case["tokens"], case["hkv"], case["dim"]), dtype=torch.float16, device="cuda")
    return s


def _prepare_append(case, gen):
    s = _prepare_tokens(case, gen)
    t, hkv, d, fmt = case["tokens"], case["hkv"], case["dim"], FORMATS[case["format"]]
    num_pages = t // PAGE + 8
    s["ks"], s["vs"] = _signs(gen, hkv, d), _signs(gen, hkv, d)
    s["slots"] = torch.randperm(num_pages * PAGE, device="cuda", generator=gen)[:t].to(torch.int32)
    if t > 256:  # a chunk fills whole pages, wherever they are
        pages = torch.randperm(num_pages, device="cuda", generator=gen)
        at = torch.arange(t, device="cuda")
        s["slots"] = (pages[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
    if own:
        s.update(_empty_pool(num_pages, hkv, d, fmt))
        s["cache"] = _handle(s, fmt, num_pages, hkv, d)
        s["k_out"] = torch.empty((t, hkv, d), dtype=torch.float16, device="cuda")
        s["v_out"] = torch.empty((t, hkv, d), dtype=torch.float16, device="cuda")
    return s


def _prepare_read(case, gen):
    t, hkv, d, fmt = case["tokens"], case["hkv"], case["dim"], FORMATS[case["format"]]
    num_pages = t // PAGE + 8
    s = {"case": case, "ks": _signs(gen, hkv, d), "vs": _signs(gen, hkv, d)}
    s.update(_pool(gen, num_pages, hkv, d, fmt, s["ks"], s["vs"]))
    pages = torch.randperm(num_pages, device="cuda", generator=gen)
    at = torch.arange(t, device="cuda") + 5  # from the middle of a page
    s["slots"] = (pages[at // PAGE] * PAGE + at % PAGE).to(torch.int32)
    if own:
        s["cache"] = _handle(s, fmt, num_pages, hkv, d)
        s["k_out"] = torch.empty((t, hkv, d), dtype=torch.float16, device="cuda")
        s["v_out"] = torch.empty((t, hkv, d), dtype=torch.float16, device="cuda")
    return s


def _shared_plan(case, gen):
    """Where the groups begin, and the prefix and continuation lengths (host)."""
    b, n = case["batch"], min(case["groups"], case["batch"])
    cpu = torch.Generator().manual_seed(int(torch.randint(0, 1 << 30, (1,), device="cuda", generator=gen)))
    if n == 1:
        offsets, prefix = [0, b], [case["prefix"]]
    else:
        cuts = sorted((torch.randperm(b - 1, generator=cpu)[:n - 1] + 1).tolist())
        offsets = [0] + cuts + [b]
        prefix = [case["prefix"]] + [max(1, int(case["prefix"] * f))
                                     for f in torch.rand(n - 1, generator=cpu).tolist()]
    suffix = torch.randint(0, case["suffix"] + 1, (b,), generator=cpu).tolist()
    suffix[0] = case["suffix"]
    return offsets, prefix, suffix


def _prepare_shared(case, gen):
    b, hq, hkv, d, fmt = case["batch"], case["hq"], case["hkv"], case["dim"], FORMATS[case["format"]]
    s = {"case": case, "ks": _signs(gen, hkv, d), "vs": _signs(gen, hkv, d)}
    offsets, prefix, suffix = _shared_plan(case, gen)
    n = len(prefix)
    prefix_pages, suffix_pages = -(-max(prefix) // PAGE), -(-max(suffix) // PAGE)
    num_pages = n * prefix_pages + b * suffix_pages
    s.update(_pool(gen, num_pages, hkv, d, fmt, s["ks"], s["vs"]))
    pages = torch.randperm(num_pages, device="cuda", generator=gen).to(torch.int32)
    s["prefix_table"] = pages[:n * prefix_pages].reshape(n, prefix_pages).contiguous()
    s["suffix_table"] = pages[n * prefix_pages:].reshape(b, suffix_pages).contiguous()
    s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    s["suffix_lens"] = torch.tensor(suffix, dtype=torch.int32, device="cuda")
    s["offsets"] = offsets
    s["q"] = torch.randn((b, hq, d), device="cuda", generator=gen).half()
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        s["cache"] = _handle(s, fmt, num_pages, hkv, d)
        s["prefix"] = [kvq.TierView(s["cache"], s["prefix_table"], s["prefix_lens"])]
        s["suffix"] = [kvq.TierView(s["cache"], s["suffix_table"], s["suffix_lens"])]
        s["out"] = torch.empty((b, hq, d), dtype=torch.float16, device="cuda")
        need = kvq.kvq_decode_shared_workspace_size(s["prefix"], offsets, s["suffix"], b, hq)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return {"rope": _run_rope, "append": _run_append, "read": _run_read, "shared": _run_shared}[s["case"]["op"]](s)


def _turn(x, cos, sin, rot, layout):
    """Rotary positions of x [tokens, heads, d] in 32 bits; cos and sin [tokens, 1, rot / 2]."""
    x = x.float()
    head, tail = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, tail], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), tail], -1)


def _cos_sin(s):
    angle = s["positions"].double()[:, None, None] * s["w"]  # 64 bits: far positions turn many times
    return (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()


def _run_rope(s):
    c = s["case"]
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        kvq.kvq_rope_apply(s["rope"], s["positions"], s["q"], s["k"], s["q_out"], s["k_out"], transpose=c["grad"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cos, sin = _cos_sin(s)
    sin = -sin if c["grad"] else sin
    return {"q": _turn(s["q"], cos, sin, c["rot"], c["layout"]).half(),
            "k": _turn(s["k"], cos, sin, c["rot"], c["layout"]).half()}


def _run_append(s):
    c = s["case"]
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        cache = s["cache"].struct
        kvq.kvq_rope_append(cache, s["rope"], s["positions"], s["k"], s["v"], s["slots"], s["q"], s["q_out"])
        kvq.kvq_dequantize(cache, s["slots"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    fmt, d = FORMATS[c["format"]], c["dim"]
    cos, sin = _cos_sin(s)
    k = _rotate(_turn(s["k"], cos, sin, c["rot"], c["layout"]), s["ks"])
    v = _rotate(s["v"], s["vs"])
    k = _decode(*_encode(k, fmt[0], fmt[2]), d, fmt[0], fmt[2])
    v = _decode(*_encode(v, fmt[1], fmt[3]), d, fmt[1], fmt[3])
    return {"q": _turn(s["q"], cos, sin, c["rot"], c["layout"]).half(), "k": _unrotate(k, s["ks"]).half(),
            "v": _unrotate(v, s["vs"]).half()}


def _stored(s, side, slots, dtype=torch.float32):
    """Tokens of the pool as the vectors that they stand for: [..., kv heads, d]."""
    c = s["case"]
    fmt, d = FORMATS[c["format"]], c["dim"]
    i = 0 if side == "k" else 1
    page, off = (slots // PAGE).long(), (slots % PAGE).long()
    rows = s[side + "_rows"][page, :, off]
    aux = s[side + "_aux"]
    aux = None if aux is None else aux[page, :, off]
    return _unrotate(_decode(rows, aux, d, fmt[i], fmt[2 + i], dtype), s[side + "s"], dtype)


def _run_read(s):
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        kvq.kvq_dequantize(s["cache"].struct, s["slots"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"k": _stored(s, "k", s["slots"]).half(), "v": _stored(s, "v", s["slots"]).half()}


def _paged(table, length):
    """Pool slots of the first `length` tokens of every row of a block table."""
    t = torch.arange(length, device="cuda")
    return table[:, t // PAGE] * PAGE + (t % PAGE).to(torch.int32)


def _run_shared(s):
    c = s["case"]
    if own:
        import quantized_decode_attention_rht_gb300 as kvq
        kvq.kvq_decode_attention_shared(s["prefix"], s["offsets"], s["suffix"], s["q"], s["out"], s["workspace"])
        return s["out"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["dim"]
    g, n = hq // hkv, len(s["offsets"]) - 1
    q = s["q"].float().view(b, hkv, g, d) / math.sqrt(d)
    # the prefix, once for every group: its sequences' queries side by side
    offsets = torch.tensor(s["offsets"], device="cuda")
    most = max(y - x for x, y in zip(s["offsets"], s["offsets"][1:]))
    member = torch.minimum(offsets[:-1, None] + torch.arange(most, device="cuda"), offsets[1:, None] - 1)
    slots = _paged(s["prefix_table"], s["prefix_table"].shape[1] * PAGE)
    k, v = _stored(s, "k", slots), _stored(s, "v", slots)  # [n, l, hkv, d]
    qp = q[member].permute(0, 2, 1, 3, 4).reshape(n, hkv, most * g, d)
    sp = qp @ k.permute(0, 2, 3, 1)
    away = torch.arange(k.shape[1], device="cuda")[None, :] >= s["prefix_lens"][:, None]
    sp = sp.masked_fill_(away[:, None, None, :], -math.inf)
    mp = sp.amax(-1, keepdim=True)
    ep = torch.exp(sp.sub_(mp))
    op, lp = ep @ v.permute(0, 2, 1, 3), ep.sum(-1, keepdim=True)
    del sp, ep, k, v
    # back to the sequences
    at = torch.arange(b, device="cuda")
    group = torch.bucketize(at, offsets[1:], right=True)
    place = at - offsets[group]
    mp, op, lp = (x.view(n, hkv, most, g, -1).permute(0, 2, 1, 3, 4)[group, place] for x in (mp, op, lp))
    # each sequence's continuation
    slots = _paged(s["suffix_table"], s["suffix_table"].shape[1] * PAGE)
    k, v = _stored(s, "k", slots).permute(0, 2, 1, 3), _stored(s, "v", slots).permute(0, 2, 1, 3)
    ss = q @ k.transpose(-1, -2)
    away = torch.arange(k.shape[2], device="cuda")[None, :] >= s["suffix_lens"][:, None]
    ss = ss.masked_fill(away[:, None, None, :], -math.inf)
    m = torch.maximum(mp, ss.amax(-1, keepdim=True))
    es, fp = torch.exp(ss - m), torch.exp(mp - m)
    return ((op * fp + es @ v) / (lp * fp + es.sum(-1, keepdim=True))).reshape(b, hq, d).half()


# --------------------------------------------------------------------------- work
def _row_bytes(name, bits, d):
    return {"fp16": 2 * d, "fp8_e4m3": d, "int4_g32": d // 2 + d // 16, "codebook": d * bits // 8 + 2}[name]


def _token_bytes(case):
    """Bytes of one cached token of one kv head."""
    fmt, d = FORMATS[case["format"]], case["dim"]
    return _row_bytes(fmt[0], fmt[2], d) + _row_bytes(fmt[1], fmt[3], d)


def work(case):
    d, hkv = case["dim"], case["hkv"]
    if case["op"] == "shared":
        gen = torch.Generator(device="cuda").manual_seed(0)
        _signs(gen, hkv, d), _signs(gen, hkv, d)
        offsets, prefix, suffix = _shared_plan(case, gen)  # of one seed: the lengths vary a little with it
        rows = hkv * _token_bytes(case)
        cached = sum(prefix) + sum(suffix)
        pairs = sum((y - x) * p for x, y, p in zip(offsets, offsets[1:], prefix)) + sum(suffix)
        return {"bytes": cached * rows + 4 * (cached // PAGE + len(suffix)) + 4 * case["batch"] * case["hq"] * d,
                "flops": 4.0 * pairs * case["hq"] * d}
    t = case["tokens"]
    if case["op"] == "read":
        return {"bytes": t * (4 + hkv * (_token_bytes(case) + 4 * d)), "flops": 2.0 * t * hkv * d * (math.log2(d) + 1)}
    turned = 3.0 * case["rot"]
    if case["op"] == "rope":
        return {"bytes": t * (4 + 4 * d * (case["hq"] + hkv)) + 4 * case["rot"],
                "flops": t * (case["hq"] + hkv) * turned}
    # q read and written, k and v read, the rows written and read back, k and v as vectors written
    return {"bytes": t * (12 + 4 * d * case["hq"] + hkv * (2 * _token_bytes(case) + 8 * d)) + 4 * case["rot"],
            "flops": t * ((case["hq"] + hkv) * turned + 4.0 * hkv * d * (math.log2(d) + 1))}


# --------------------------------------------------------------------------- 64 bits
def _exact_turn(x, positions, case, transpose=False):
    """Each pair as a complex number, multiplied by the scaled unit number of its angle."""
    rot = case["rot"]
    w, scale = _frequencies(rot, case["scaling"])
    angle = torch.outer(positions.double(), torch.from_numpy(w).cuda()) * (-1.0 if transpose else 1.0)
    unit = torch.polar(torch.full_like(angle, scale), angle)[:, None, :]
    y = x.double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot].clone()) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)) * unit
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_butterflies(x):
    """Walsh-Hadamard transform of the last axis / sqrt(d), in 64 bits."""
    d = x.shape[-1]
    y, step = x.double(), 1
    while step < d:
        y = y.reshape(*x.shape[:-1], d // (2 * step), 2, step)
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        step *= 2
    return y / math.sqrt(d)


def _exact_quantised(x, fmt, bits):
    """The vectors that the stored form of rotated vectors x (64 bits) stands for."""
    d = x.shape[-1]
    if fmt == "fp16":
        return x.float().half().double()
    if fmt == "fp8_e4m3":
        m = x.abs().clamp(min=2.0 ** -9, max=448.0)
        step = 2.0 ** (torch.floor(torch.log2(m)).clamp(min=-6.0) - 3.0)
        return (torch.round(x / step) * step).clamp(-448.0, 448.0)
    if fmt == "int4_g32":
        g = x.reshape(*x.shape[:-1], d // 32, 32)
        scale = (g.abs().amax(-1, keepdim=True) / 7.0).half().double()
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        return (torch.round(g / safe).clamp(-7.0, 7.0) * scale).reshape(x.shape)
    cent, bounds = (torch.from_numpy(t).cuda().double() for t in _table(bits))
    norm = x.norm(dim=-1, keepdim=True)
    u = x * (math.sqrt(d) / torch.where(norm > 0, norm, torch.ones_like(norm)))
    codes = sum((u > bound).long() for bound in bounds)
    return cent[codes] * norm.half().double() / math.sqrt(d)


def _exact_stored(s, side, slots, case):
    """Cached tokens in 64 bits, their bits taken apart one field at a time."""
    fmt, bits = FORMATS[case["format"]][0 if side == "k" else 1], FORMATS[case["format"]][2 if side == "k" else 3]
    d = case["dim"]
    page, off = torch.div(slots, PAGE, rounding_mode="floor").long(), slots.long() % PAGE
    rows = s[side + "_rows"].transpose(1, 2)[page, off]
    aux = s[side + "_aux"]
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
    return _exact_butterflies(x) * s[side + "s"].double()


def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    if case["op"] == "rope":
        return {x: _exact_turn(s[x], s["positions"], case, case["grad"]) for x in ("q", "k")}
    if case["op"] == "append":
        fmt = FORMATS[case["format"]]
        k = _exact_butterflies(_exact_turn(s["k"], s["positions"], case) * s["ks"].double())
        v = _exact_butterflies(s["v"].double() * s["vs"].double())
        return {"q": _exact_turn(s["q"], s["positions"], case),
                "k": _exact_butterflies(_exact_quantised(k, fmt[0], fmt[2])) * s["ks"].double(),
                "v": _exact_butterflies(_exact_quantised(v, fmt[1], fmt[3])) * s["vs"].double()}
    if case["op"] == "read":
        return {x: _exact_stored(s, x, s["slots"], case) for x in ("k", "v")}
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["dim"]
    out = torch.empty((b, hq, d), dtype=torch.float64, device="cuda")

    def tokens(table, length):
        t = torch.arange(length, device="cuda")
        slots = table.long()[t // PAGE] * PAGE + t % PAGE
        return [_exact_stored(s, x, slots, case).transpose(0, 1) for x in ("k", "v")]

    prefix, suffix = s["prefix_lens"].tolist(), s["suffix_lens"].tolist()
    for i, (first, last) in enumerate(zip(s["offsets"], s["offsets"][1:])):
        pk, pv = tokens(s["prefix_table"][i], prefix[i])
        for r in range(first, last):
            sk, sv = tokens(s["suffix_table"][r], suffix[r])
            k, v = torch.cat([pk, sk], 1), torch.cat([pv, sv], 1)
            q = s["q"][r].double().reshape(hkv, hq // hkv, d)
            p = torch.softmax(torch.bmm(q, k.transpose(1, 2)) / math.sqrt(d), -1)
            out[r] = torch.bmm(p, v).reshape(hq, d)
    return out
