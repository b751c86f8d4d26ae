"""The attention layer between delta-rule layers, as cases to be measured: rotary positions (with several axes) and
head norms fused with the write of a paged key-value cache, its read-back, and attention over the cache for decoded
tokens and for prompts.

With `own` false, run() computes them from elementary torch operations; with `own` true it calls the package's entry
points.  exact() computes the same outputs in 64 bits from the definitions.

A cache is a pool of pages of `page` tokens; table[i] lists the pages of sequence i.  A page holds, for each key head, a
block of page * d values in units of 16 bytes (8 bf16 values, or 16 int8 codes; behind the codes a float scale per
token).  A unit of keys has values of one token, the units ordered [d / unit][page]; a unit of values has one dimension
of as many tokens, the units ordered [page / unit][d].  The new tokens of sequence i are rows starts[i] .. starts[i + 1]
of q, k, v and out, and the last ones of its lens[i] tokens.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 1e6


# ---- cases --------------------------------------------------------------------

# "lens": for each sequence its new tokens + those that the cache holds already
def listed():
    return [
        # one decoded token on its way into the cache: all latency
        {"name": "cache one token", "op": "cache", "lens": "1+700", "hq": 32, "hk": 8, "d": 128, "rot": 128, "axes": 1,
         "norm": False, "bits": 16, "page": 64},
        # prompts with images (three axes, part of each head rotated, heads normed) into an int8 cache, and read back:
        # one token, none, odd lengths, prompts continued inside a page
        {"name": "cache ragged", "op": "cache", "lens": "1+37 700+0 65+1000 0+5 1300+129 64+64", "hq": 16, "hk": 2, "d": 256,
         "rot": 64, "axes": 3, "norm": True, "bits": 8, "page": 16},
        # one long prompt
        {"name": "cache prompt", "op": "cache", "lens": "8192+0", "hq": 32, "hk": 8, "d": 128, "rot": 128, "axes": 1,
         "norm": True, "bits": 16, "page": 64},
        # one token of a short conversation: all latency
        {"name": "decode one token", "op": "decode", "lens": "1+700", "hq": 32, "hk": 8, "d": 128, "bits": 16, "page": 64,
         "window": 0, "cap": 0.0},
        # one token behind a long document, the cache in int8
        {"name": "decode long", "op": "decode", "lens": "1+130000", "hq": 32, "hk": 8, "d": 128, "bits": 8, "page": 64,
         "window": 0, "cap": 0.0},
        # a batch in the middle of its answers, of lengths from a few tokens to 8192, small pages
        {"name": "decode batch", "op": "decode", "batch": 64, "new": 1, "longest": 8192, "hq": 32, "hk": 8, "d": 128, "bits": 16,
         "page": 16, "window": 0, "cap": 0.0},
        # four drafted tokens of each of eight sequences verified together, wide heads, capped scores
        {"name": "decode verify", "op": "decode", "batch": 8, "new": 4, "longest": 16384, "hq": 16, "hk": 2, "d": 256, "bits": 8,
         "page": 64, "window": 0, "cap": 50.0},
        # a layer with a sliding window, every head with its own keys, a head size that is no power of two
        {"name": "decode window", "op": "decode", "batch": 96, "new": 1, "longest": 5000, "hq": 12, "hk": 12, "d": 80, "bits": 16,
         "page": 32, "window": 1024, "cap": 0.0},
        # one prompt
        {"name": "prompt", "op": "prompt", "lens": "2048+0", "hq": 32, "hk": 8, "d": 128, "bits": 16, "page": 64, "window": 0,
         "cap": 0.0},
        # packed prompts of ragged lengths, some continued, over an int8 cache in small pages
        {"name": "prompt ragged", "op": "prompt", "lens": "1+0 700+0 65+1000 0+300 1300+2000 64+64 129+4000 63+1", "hq": 32,
         "hk": 8, "d": 128, "bits": 8, "page": 16, "window": 0, "cap": 0.0},
        # a prompt through a layer with a sliding window and capped scores, wide heads
        {"name": "prompt window", "op": "prompt", "lens": "6001+0", "hq": 16, "hk": 2, "d": 256, "bits": 16, "page": 64,
         "window": 1024, "cap": 30.0},
        # the last part of a long prompt that is taken in parts
        {"name": "prompt part", "op": "prompt", "lens": "4096+12288", "hq": 32, "hk": 8, "d": 128, "bits": 16, "page": 64,
         "window": 0, "cap": 0.0},
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; the larger sizes odd, as the listed ones are mostly round."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - 1 if n > 2048 and n % 2 == 0 else n


def draw(rng):
    op = rng.choice(["cache", "decode", "decode", "prompt", "prompt"])
    d = rng.choice([64, 80, 96, 128, 128, 256])
    hk = rng.choice([h for h in (1, 2, 4, 8, 12) if h * d <= 1024])
    hq = hk * rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if g * hk * d <= 4096])
    c = {"op": op, "hq": hq, "hk": hk, "d": d, "bits": rng.choice([8, 16]), "page": rng.choice([16, 32, 64, 128])}
    if op == "decode":
        batch = _log(rng, 1, 64)
        return {**c, "batch": batch, "new": rng.choice([1, 1, 1, 2, 3, 4, 8]), "longest": _log(rng, 1, min(130000, 524288 // batch)),
                "window": rng.choice([0, 0, 0, 100, 1024]), "cap": rng.choice([0.0, 0.0, 30.0])}
    count = rng.choice([1, 1, 2, 3, 5, 8])
    if op == "cache":
        new = [_log(rng, 1, 8192 // count) for _ in range(count)]
        old = [rng.choice([0, _log(rng, 1, 2000)]) for _ in range(count)]
        c.update(rot=rng.choice([d, d, d // 32 * 16]), axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.5)
    else:
        new = [_log(rng, 1, 4096 // count) for _ in range(count)]
        old = [rng.choice([0, _log(rng, 1, 12288 // count)]) for _ in range(count)]
        c.update(window=rng.choice([0, 0, 0, 100, 1024]), cap=rng.choice([0.0, 0.0, 30.0]))
    return {**c, "lens": " ".join("%d+%d" % p for p in zip(new, old))}


def _sequences(case):
    """For each sequence its new tokens and all of its tokens."""
    if "lens" in case:
        pairs = [p.split("+") for p in case["lens"].split()]
        return [int(n) for n, _ in pairs], [int(n) + int(c) for n, c in pairs]
    # lengths spread evenly up to the longest, in no order
    new = [case["new"]] * case["batch"]
    return new, [n + int(case["longest"] * math.fmod(0.75 + 0.6180339887498949 * i, 1.0)) for i, n in enumerate(new)]


# ---- inputs ---------------------------------------------------------------------

def _cache(case, pages, normal, codes, uniform):
    """A pool of pages with values in every place, as bytes."""
    rows = pages * case["hk"]
    values = case["page"] * case["d"]
    if case["bits"] == 16:
        return normal(rows, values).view(torch.uint8).view(-1)
    buf = torch.empty(rows, values + 4 * case["page"], dtype=torch.uint8, device=DEV)
    buf[:, :values] = codes(rows, values).view(torch.uint8)
    buf[:, values:] = ((0.5 + uniform(rows, case["page"])) / 60.0).view(torch.uint8)
    return buf.view(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV, dtype=torch.float32)

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    new, lens = _sequences(case)
    tokens, count = sum(new), len(new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    width = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = [0]
    for n in used:
        at.append(at[-1] + n)
    places = torch.arange(width, device=DEV)
    first, held = torch.tensor(at[:-1], device=DEV), torch.tensor(used, device=DEV)
    # entries behind a sequence's last page point anywhere in the pool
    table = order[(first[:, None] + torch.minimum(places, held[:, None])) % pages].contiguous()
    s = {"case": case, "tokens": tokens, "new": new, "lens_list": lens, "starts": ints(starts), "lens": ints(lens), "table": table,
         "k_cache": _cache(case, pages, normal, codes, uniform), "v_cache": _cache(case, pages, normal, codes, uniform)}
    # where each packed token belongs: its sequence, its place there, its place among the sequence's new tokens
    s["seq"] = torch.repeat_interleave(torch.arange(count, device=DEV), torch.tensor(new, device=DEV), output_size=tokens)
    s["index"] = torch.arange(tokens, device=DEV) - s["starts"][:-1].long()[s["seq"]]
    s["pos"] = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()[s["seq"]] + s["index"]
    packed = normal(tokens, (hq + 2 * hk) * d + 16)  # q, k, v and what else the projection leaves in a row
    s["q"] = packed[:, :hq * d].unflatten(1, (hq, d))
    s["out"] = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device=DEV)
    if case["op"] == "cache":
        s["k"] = packed[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = packed[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
        s["q_norm"] = (1 + 0.2 * normal(d)) if case["norm"] else None
        s["k_norm"] = (1 + 0.2 * normal(d)) if case["norm"] else None
        half = case["rot"] // 2
        angle = torch.arange(max(lens) + 64, device=DEV, dtype=torch.float64)[:, None] * THETA ** (
            -torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["cos_sin"] = torch.stack([torch.cos(angle), torch.sin(angle)], 1).float().contiguous()
        s["positions"] = s["axis"] = None
        if case["axes"] > 1:  # images: rows and columns of patches, frequencies of the axes in turn
            s["positions"] = torch.stack([s["pos"], s["pos"] // 24 + 7, s["pos"] % 24 + 7]).to(torch.int32).contiguous()
            s["axis"] = (torch.arange(half, device=DEV) % case["axes"]).to(torch.uint8)
        s["k_back"] = torch.empty(tokens, hk, d, dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.empty_like(s["k_back"])
    if case["op"] == "decode":
        s["workspace"] = torch.empty(workspace_bytes(tokens, hq, d), dtype=torch.uint8, device=DEV)
    return s


def workspace_bytes(tokens, hq, d):
    """An upper bound of what paged_attention_decode asks for."""
    return (128 << 20) + 16 * tokens * hq * (d + 4)


# ---- one pass ---------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "cache":
        return (_own_cache if own else _plain_cache)(s)
    if own:
        return (_own_decode if op == "decode" else _own_prompt)(s)
    return _plain_attention(s)


def _own_cache(s):
    import bit_quantized_matmul_quantize_amd as bq
    c = s["case"]
    bq.rope_write_kv_cache(s["q"], s["k"], s["v"], s["out"], s["k_cache"], s["v_cache"], s["starts"], s["lens"], s["table"],
                           c["page"], c["bits"], cos_sin=s["cos_sin"], positions=s["positions"], axis=s["axis"],
                           q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    if c["bits"] == 16:
        return {"q": s["out"], "k": s["k_cache"].view(torch.bfloat16), "v": s["v_cache"].view(torch.bfloat16)}
    bq.read_kv_cache(s["k_cache"], s["v_cache"], s["k_back"], s["v_back"], s["starts"], s["lens"], s["table"], c["page"], c["bits"])
    return {"q": s["out"], "k": s["k_back"], "v": s["v_back"]}


def _own_decode(s):
    import bit_quantized_matmul_quantize_amd as bq
    c = s["case"]
    bq.paged_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["out"], s["starts"], s["lens"], s["table"], s["workspace"],
                              c["hk"], c["page"], c["bits"], window=c["window"], cap=c["cap"])
    return s["out"]


def _own_prompt(s):
    import bit_quantized_matmul_quantize_amd as bq
    c = s["case"]
    bq.paged_attention_prefill(s["q"], s["k_cache"], s["v_cache"], s["out"], s["starts"], s["lens"], s["table"],
                               c["hk"], c["page"], c["bits"], window=c["window"], cap=c["cap"])
    return s["out"]


def _views(case, buf, keys):
    """The units of a cache as [pages, hk, d / unit, page, unit] (keys) or [pages, hk, page / unit, d, unit], and an int8
    cache's scales [pages, hk, page]."""
    hk, d, page = case["hk"], case["d"], case["page"]
    unit = 8 if case["bits"] == 16 else 16
    shape = (d // unit, page, unit) if keys else (page // unit, d, unit)
    if case["bits"] == 16:
        return buf.view(torch.bfloat16).view(-1, hk, *shape), None
    blocks = buf.view(-1, hk, page * (d + 4))
    return blocks[:, :, :page * d].view(torch.int8).unflatten(2, shape), blocks[:, :, page * d:].view(torch.float32)


def _plain_cache(s):
    c = s["case"]
    hk, d, page, rot = c["hk"], c["d"], c["page"], c["rot"]
    unit, half = 8 if c["bits"] == 16 else 16, rot // 2
    if c["axes"] == 1:
        row = s["cos_sin"][s["pos"]]
        cos, sin = row[:, None, 0], row[:, None, 1]
    else:
        f = torch.arange(half, device=DEV)
        row = s["cos_sin"][s["positions"].long()[s["axis"].long()].t(), :, f]
        cos, sin = row[:, None, :, 0], row[:, None, :, 1]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
        a, b, rest = x.split([half, half, d - rot], dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    s["out"].copy_(turned(s["q"], s["q_norm"]))
    k, v = turned(s["k"], s["k_norm"]), s["v"].float()
    (kc, ks), (vc, vs) = _views(c, s["k_cache"], True), _views(c, s["v_cache"], False)
    at, off = s["table"].long()[s["seq"], s["pos"] // page], s["pos"] % page
    if c["bits"] == 16:
        kc[at, :, :, off] = k.bfloat16().unflatten(2, (d // unit, unit))
        vc[at, :, off // unit, :, off % unit] = v.bfloat16()
        return {"q": s["out"], "k": s["k_cache"].view(torch.bfloat16), "v": s["v_cache"].view(torch.bfloat16)}

    def quantized(x):
        top = x.abs().amax(2, keepdim=True)
        codes = torch.round(127.0 * x.double() / top)
        return torch.where(top > 0, codes, 0.0).to(torch.int8), top[:, :, 0] / 127.0

    (kq, kt), (vq, vt) = quantized(k), quantized(v)
    kc[at, :, :, off] = kq.unflatten(2, (d // unit, unit))
    vc[at, :, off // unit, :, off % unit] = vq
    ks[at, :, off], vs[at, :, off] = kt, vt
    s["k_back"].copy_(kc[at, :, :, off].flatten(2).float() * ks[at, :, off][..., None])
    s["v_back"].copy_(vc[at, :, off // unit, :, off % unit].float() * vs[at, :, off][..., None])
    return {"q": s["out"], "k": s["k_back"], "v": s["v_back"]}


def _rows(case, buf, keys, table):
    """The cache's rows of every sequence, in 32 bits: [sequence, hk, place, d]."""
    units, scales = _views(case, buf, keys)
    x = units[table].float()  # [sequence, page, hk, d / unit, offset, unit] or [sequence, page, hk, offset / unit, d, unit]
    x = x.permute(0, 2, 1, 4, 3, 5) if keys else x.permute(0, 2, 1, 3, 5, 4)
    x = x.reshape(table.shape[0], case["hk"], -1, case["d"])
    if scales is None:
        return x
    return x * scales[table].permute(0, 2, 1, 3).reshape(table.shape[0], case["hk"], -1, 1)


def _plain_attention(s):
    """All sequences side by side, padded to the longest; the heads of a key head are rows of one product."""
    c = s["case"]
    hq, hk, d, count, most = c["hq"], c["hk"], c["d"], len(s["new"]), max(s["new"])
    g, table = hq // hk, s["table"].long()
    q = torch.zeros(count, most, hq, d, device=DEV)
    q[s["seq"], s["index"]] = s["q"].float()
    q = q.view(count, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(count, hk, g * most, d)
    k = _rows(c, s["k_cache"], True, table)
    scores = (q @ k.transpose(2, 3)) * d ** -0.5
    if c["cap"]:
        scores = torch.tanh(scores / c["cap"]) * c["cap"]
    scores = scores.view(count, hk, g, most, -1)
    n = s["starts"][1:] - s["starts"][:-1]
    here = (s["lens"] - n)[:, None] + torch.arange(most, device=DEV)  # positions of the rows
    at = torch.arange(scores.shape[-1], device=DEV)
    seen = at <= here[..., None]
    if c["window"]:
        seen &= at > here[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = torch.exp_(scores)
    total = p.sum(-1, keepdim=True)
    v = _rows(c, s["v_cache"], False, table)
    o = (p.view(count, hk, g * most, -1) @ v).view(count, hk, g, most, d) / total
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[s["seq"], s["index"]].reshape(s["out"].shape))
    return s["out"]


# ---- what one pass cannot do without --------------------------------------------------

def work(case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    new, lens = _sequences(case)
    tokens, size = sum(new), 2.0 if case["bits"] == 16 else 1.0 + 4.0 / d  # bytes of a value in the cache
    if case["op"] == "cache":
        # q, k, v in, q out, k and v into the cache; from an int8 cache read back: codes in, bf16 out
        values = 4 * hq + 2 * hk * (2 + size) + (2 * hk * (size + 2) if case["bits"] == 8 else 0)
        return {"bytes": tokens * (values * d + 4 * case["rot"]),
                "flops": tokens * (hq + hk) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    pairs = held = 0
    for n, length in zip(new, lens):
        if n == 0:
            continue
        window = case["window"] or length
        first = length - n  # position p sees min(p + 1, window) keys
        full = max(0, min(n, window - first))  # tokens that see all before them
        pairs += full * first + full * (full + 1) // 2 + (n - full) * window
        held += length - max(0, first + 1 - window)
    return {"bytes": 2 * held * hk * d * size + 4 * tokens * hq * d, "flops": 4 * pairs * hq * d}


# ---- the definitions, in 64 bits ------------------------------------------------------

def _place(s, i, p):
    """Page and offset of the places p of sequence i."""
    page = s["case"]["page"]
    return s["table"][i].long()[p // page], p % page


def _exact_rows(s, i, p, head, keys):
    """Rows [place, d] of one key head, value by value from their bytes."""
    c = s["case"]
    d, page = c["d"], c["page"]
    at, off = _place(s, i, p)
    at, off, j = at[:, None], off[:, None], torch.arange(d, device=DEV)[None]
    unit = 8 if c["bits"] == 16 else 16
    inside = (j // unit * page + off) * unit + j % unit if keys else (off // unit * d + j) * unit + off % unit
    buf = s["k_cache" if keys else "v_cache"]
    if c["bits"] == 16:
        return buf.view(torch.bfloat16)[(at * c["hk"] + head) * page * d + inside].double()
    block = (at * c["hk"] + head) * page * (d + 4)
    return buf.view(torch.int8)[block + inside].double() * buf.view(torch.float32)[(block + page * d) // 4 + off].double()


def exact(case, seed):
    s = prepare(case, seed)
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    if case["op"] != "cache":
        out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device=DEV)
        t0 = 0
        for i, (n, length) in enumerate(zip(s["new"], s["lens_list"])):
            for h in range(hq if n else 0):
                low = max(0, length - n + 1 - case["window"]) if case["window"] else 0
                p = torch.arange(low, length, device=DEV)
                if h % (hq // hk) == 0:
                    keys, values = (_exact_rows(s, i, p, h // (hq // hk), w) for w in (True, False))
                x = s["q"][t0:t0 + n, h].double() @ keys.t() / math.sqrt(d)
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                mine = torch.arange(length - n, length, device=DEV)[:, None]
                hidden = p > mine
                if case["window"]:
                    hidden |= mine - p >= case["window"]
                out[t0:t0 + n, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ values
            t0 += n
        return out
    half = case["rot"] // 2
    angles = s["positions"].long() if case["axes"] > 1 else s["pos"][None]
    which = s["axis"].tolist() if case["axes"] > 1 else [0] * half

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * weight.double()
        y = x.clone()
        for f in range(half):
            c, z = (s["cos_sin"][angles[which[f]], w, f].double()[:, None] for w in (0, 1))
            y[:, :, f] = x[:, :, f] * c - x[:, :, f + half] * z
            y[:, :, f + half] = x[:, :, f + half] * c + x[:, :, f] * z
        return y

    q, k, v = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"]), s["v"].double()
    if case["bits"] == 8:
        def stepped(x):
            step = x.abs().max(2, keepdim=True).values / 127
            return torch.round(x / step) * step
        return {"q": q, "k": stepped(k), "v": stepped(v)}
    kc, vc = s["k_cache"].view(torch.bfloat16).double(), s["v_cache"].view(torch.bfloat16).double()
    at, off = s["table"].long()[s["seq"], s["pos"] // page][:, None, None], (s["pos"] % page)[:, None, None]
    h, j = torch.arange(hk, device=DEV)[None, :, None], torch.arange(d, device=DEV)
    kc[(at * hk + h) * page * d + (j // 8 * page + off) * 8 + j % 8] = k
    vc[(at * hk + h) * page * d + (off // 8 * d + j) * 8 + off % 8] = v
    return {"q": q, "k": kc, "v": vc}
