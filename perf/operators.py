"""The operators around the quantized projections, as cases to be measured: the RMS norm with the
residual's addition and an 8-bit output, the int8 matrix product with a scale per token and per
channel, and the gated delta rule in its chunked (prefill) and recurrent (decode) forms.

With `own` false, run() computes them from elementary torch operations; with `own` true it calls
the package's entry points.  exact() computes the same outputs in 64 bits from the definitions.
The sizes are those of the projections that the framework serves: hidden sizes 2048 and 5120, FFN
17408, a qkvz projection of 12288 rows with 16 key heads and 32 value heads of 128.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
CHUNK = 64


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # the norm before a projection of one decoded token: all latency
        {"name": "norm one token", "op": "norm", "m": 1, "k": 2048, "out": "int8", "residual": True},
        # an odd hidden size, a few dozen tokens, into the block format of the 2- and 4-bit products
        {"name": "norm ragged q8_1", "op": "norm", "m": 333, "k": 2563, "out": "q8_1", "residual": True},
        # the norm before the FFN of a prompt of 4096 tokens
        {"name": "norm prompt", "op": "norm", "m": 4096, "k": 5120, "out": "int8", "residual": True},
        # the qkvz projection of one decoded token: reads the whole weight for one row
        {"name": "product one token", "op": "product", "m": 1, "n": 12288, "k": 2048, "bias": False},
        # the FFN's down projection of a verified batch of eight tokens: a long sum, few rows
        {"name": "product verify", "op": "product", "m": 8, "n": 5120, "k": 17408, "bias": False},
        # odd in every size, with a bias: a short prompt through a layer whose sizes are no tile's
        {"name": "product ragged", "op": "product", "m": 333, "n": 4133, "k": 2563, "bias": True},
        # the FFN's gate projection of a prompt of 4096 tokens: the largest matrix product
        {"name": "product prompt", "op": "product", "m": 4096, "n": 17408, "k": 5120, "bias": False},
        # one prompt of 2048 tokens through the delta rule, from an empty state
        {"name": "delta prompt", "op": "chunked", "lens": "2048", "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "l2norm": True, "fresh": True},
        # packed prompts of ragged lengths (one token, none, one beyond a chunk), continued from states
        {"name": "delta ragged", "op": "chunked", "lens": "1 700 65 0 1300 64 129 63", "hk": 16, "hv": 32, "dk": 128,
         "dv": 128, "l2norm": True, "fresh": False},
        # one long document
        {"name": "delta long", "op": "chunked", "lens": "16384", "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "l2norm": True, "fresh": True},
        # one decoded token of one sequence
        {"name": "delta one token", "op": "recurrent", "batch": 1, "tokens": 1, "hk": 16, "hv": 32, "dk": 128,
         "dv": 128, "l2norm": True},
        # one decoded token of each of 96 sequences: reads and writes every state
        {"name": "delta decode batch", "op": "recurrent", "batch": 96, "tokens": 1, "hk": 16, "hv": 32, "dk": 128,
         "dv": 128, "l2norm": True},
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm; the larger sizes odd, as the listed ones are mostly round."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - 1 if n > 2048 and n % 2 == 0 else n


def draw(rng):
    op = rng.choice(["norm", "product", "chunked", "recurrent"])
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 64, 5120),
                "out": rng.choice(["int8", "q8_1", "bf16"]), "residual": rng.random() < 0.75}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 17408), "k": _log(rng, 64, 5120),
                "bias": rng.random() < 0.5}
    heads = {"hk": rng.choice([1, 2, 4, 8, 16]), "dk": rng.choice([64, 128]), "dv": rng.choice([64, 80, 128])}
    heads["hv"] = heads["hk"] * rng.choice([1, 2])
    if op == "recurrent":
        return {"op": op, "batch": _log(rng, 1, 96), "tokens": rng.choice([1, 1, 1, 2, 3, 4, 8]), **heads,
                "l2norm": rng.random() < 0.75}
    count = rng.choice([1, 1, 2, 4, 8])
    lens = [_log(rng, 1, 8192 // count) for _ in range(count)]
    lens[0] += 64
    return {"op": op, "lens": " ".join(str(n) for n in lens), **heads, "l2norm": rng.random() < 0.75,
            "fresh": rng.random() < 0.5}


# ---- inputs ---------------------------------------------------------------------

def _pad(k, to):
    return (k + to - 1) // to * to


def _int8_rows(x):
    """Rows as a program keeps its int8 weights: codes [rows][k padded to 128], then a float scale per row."""
    rows, k = x.shape
    kp = _pad(k, 128)
    scale = x.abs().amax(1) / 127.0
    buf = torch.zeros(rows * kp + 4 * rows, dtype=torch.uint8, device=DEV)
    codes = buf[:rows * kp].view(torch.int8).view(rows, kp)
    codes[:, :k] = torch.round(x / scale[:, None]).clamp_(-127, 127).to(torch.int8)
    buf[rows * kp:].view(torch.float32).copy_(scale)
    return buf


def _split_int8_rows(buf, rows, k):
    kp = _pad(k, 128)
    return buf[:rows * kp].view(torch.int8).view(rows, kp)[:, :k], buf[rows * kp:rows * kp + 4 * rows].view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV, dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        outlier = 1.0 + 19.0 * (uniform(k) < 0.01).float()  # channels far above the others
        s["x"] = (normal(m, k) * outlier).bfloat16()
        s["residual"] = (normal(m, k) * 3.0).bfloat16() if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * normal(k)).bfloat16()
        if case["out"] == "bf16":
            s["out"] = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
        else:
            kp = _pad(k, 128) if case["out"] == "int8" else _pad(k, 256)
            size = m * kp + 4 * m if case["out"] == "int8" else m * kp + m * (kp // 32) * 4
            s["out"] = torch.empty(size, dtype=torch.uint8, device=DEV)
            if case["out"] == "int8":
                s["codes"], s["scale"] = _split_int8_rows(s["out"], m, k)
                s["scale"] = s["scale"][:, None]
            else:
                s["codes"] = s["out"][:m * kp].view(torch.int8).view(m, kp // 32, 32)
                s["scale"] = s["out"][m * kp:].view(torch.float16).view(m, kp // 32, 2)[:, :, :1]
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["act"] = _int8_rows(normal(m, k))
        s["weight"] = _int8_rows(normal(n, k) * 0.02)
        s["bias"] = (normal(n) * 0.1).bfloat16() if case["bias"] else None
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    else:
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        lens = [int(n) for n in case["lens"].split()] if case["op"] == "chunked" else [case["tokens"]] * case["batch"]
        tokens, count = sum(lens), len(lens)
        # q, k, v and what else the packed projection leaves in a row
        packed = normal(tokens, 2 * hk * dk + 2 * hv * dv + 16)
        if not case["l2norm"]:  # the caller has normalised the heads of q and k
            heads = packed[:, :2 * hk * dk].view(tokens, 2 * hk, dk)
            heads /= heads.norm(dim=-1, keepdim=True)
        packed = packed.bfloat16()
        s["q"] = packed[:, :hk * dk].unflatten(1, (hk, dk))
        s["k"] = packed[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
        s["v"] = packed[:, 2 * hk * dk:2 * hk * dk + hv * dv].unflatten(1, (hv, dv))
        # the decay of a head: -A softplus(a + bias), from nearly none to forgetting in a few tokens
        step = torch.exp(uniform(hv) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        bias = step + torch.log(-torch.expm1(-step))
        s["g"] = -(0.5 + 15.5 * uniform(hv)) * torch.nn.functional.softplus(normal(tokens, hv) + bias)
        s["beta"] = torch.sigmoid(normal(tokens, hv))
        slots = count + 3
        s["state"] = normal(slots, hv, dk, dv) * 0.05
        s["slots"] = torch.randperm(slots, generator=gen, device=DEV)[:count].to(torch.int32)
        s["lens"] = lens
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(tokens, hv, dv, dtype=torch.bfloat16, device=DEV)
        if case["op"] == "chunked":
            s["fresh"] = torch.full((count,), int(case["fresh"]), dtype=torch.uint8, device=DEV)
            # room for every chunk's triangular factors and re-laid rows, as the entry point asks for
            longest = max(lens)
            at = torch.arange(longest, device=DEV)
            s["inside"] = at[None, :] < torch.tensor(lens, device=DEV)[:, None]
            s["workspace"] = torch.empty(workspace_bytes(tokens, count, hk, hv, dk), dtype=torch.uint8, device=DEV)
    return s


def workspace_bytes(tokens, count, hk, hv, dk):
    """An upper bound of what gated_delta_rule_chunked asks for: 64 KB for a chunk of a value head, and
    96 bytes for each of its 64 rows and values of a key head."""
    chunks = tokens // CHUNK + count
    return chunks * (hv * 65536 + hk * CHUNK * dk * 16) + 4096


# ---- one pass ---------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "norm":
        return (_own_norm if own else _plain_norm)(s)
    if op == "product":
        return (_own_product if own else _plain_product)(s)
    if op == "chunked":
        return (_own_chunked if own else _plain_chunked)(s)
    return (_own_recurrent if own else _plain_recurrent)(s)


def _own_norm(s):
    import bit_quantized_matmul_quantize_amd as bq
    c = s["case"]
    m, k = c["m"], c["k"]
    if c["out"] == "int8":
        bq.add_rms_norm_quantize_int8(s["x"], s["residual"], s["weight"], s["out"], m, k, EPS)
        y = s["codes"] * s["scale"]
    elif c["out"] == "q8_1":
        bq.add_rms_norm_quantize_q8_1(s["x"], s["residual"], s["weight"], s["out"], m, k, EPS)
        y = (s["codes"] * s["scale"].float()).view(m, -1)[:, :k]
    else:
        bq.add_rms_norm_bf16(s["x"], s["residual"], s["weight"], s["out"], m, k, EPS)
        y = s["out"]
    return {"y": y, "residual": s["residual"]}


def _plain_norm(s):
    c = s["case"]
    m, k = c["m"], c["k"]
    h = s["x"]
    if s["residual"] is not None:
        h = s["residual"].copy_(s["x"].float() + s["residual"].float())
    t = h.float() * s["weight"].float()
    # the mean in 64 bits, and y from it: values next to a border of the 8-bit codes
    rstd = torch.rsqrt(h.double().square().mean(1, keepdim=True) + EPS)
    if c["out"] == "int8":
        top = t.abs().amax(1, keepdim=True)
        codes = torch.round((127.0 * t).double() / top)  # 23 significant bits: exact before the division
        codes = torch.where(top > 0, codes, 0.0)
        return {"y": codes.float() * (top * rstd / 127.0).float(), "residual": s["residual"]}
    y = (t * rstd).float().bfloat16()
    if c["out"] == "q8_1":
        kp = _pad(k, 256)
        b = torch.nn.functional.pad(y.float(), (0, kp - k)).view(m, kp // 32, 32)
        d = (b.abs().amax(2, keepdim=True) / 127.0).half().float()
        q = b.abs().double() / d
        q = torch.where(d > 0, torch.floor(q + 0.5).clamp(max=127.0) * torch.sign(b), 0.0)  # halves away from zero
        y = (q.float() * d).view(m, kp)[:, :k]
    return {"y": y, "residual": s["residual"]}


def _own_product(s):
    import bit_quantized_matmul_quantize_amd as bq
    c = s["case"]
    bq.w8a8_gemm(s["act"], s["weight"], s["out"], c["m"], c["n"], c["k"], bias=s["bias"])
    return s["out"]


def _plain_product(s):
    c = s["case"]
    a, sa = _split_int8_rows(s["act"], c["m"], c["k"])
    w, sw = _split_int8_rows(s["weight"], c["n"], c["k"])
    y = a.float() @ w.float().t() * sa[:, None] * sw
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.bfloat16()


def _own_chunked(s):
    import bit_quantized_matmul_quantize_amd as bq
    bq.gated_delta_rule_chunked(s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"], s["state"], s["starts"],
                                s["workspace"], slots=s["slots"], fresh=s["fresh"], l2norm=s["case"]["l2norm"])
    return {"out": s["out"], "state": s["state"]}


def _own_recurrent(s):
    import bit_quantized_matmul_quantize_amd as bq
    bq.gated_delta_rule_recurrent(s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"], s["state"], s["starts"],
                                  slots=s["slots"], l2norm=s["case"]["l2norm"])
    return {"out": s["out"], "state": s["state"]}


def _unit(x, l2norm):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) if l2norm else x


def _unit_inverse(lower):
    """(1 + lower)^-1 for strictly lower triangles: blocks of 1, 2, 4, ... along the diagonal are joined in
    pairs, inverse([[a, 0], [c, b]]) = [[a', 0], [-b' c a', b']]."""
    inverse, at = torch.eye(CHUNK, device=DEV).expand_as(lower), torch.arange(CHUNK, device=DEV)
    for size in (1, 2, 4, 8, 16, 32):
        pair = (at[:, None] // (2 * size) == at // (2 * size)) & (at[:, None] // size != at // size)
        inverse = inverse - inverse @ (lower * pair) @ inverse
    return inverse


def _plain_chunked(s):
    """In chunks of 64 tokens: within a chunk products and a triangular inverse, all chunks at once; from
    chunk to chunk the state.  The packed sequences are laid out as [sequence, chunk, head, token, value];
    tokens past a sequence's end have a zero gate, key, value and decay."""
    c = s["case"]
    count, hk, hv, dk, dv = len(s["lens"]), c["hk"], c["hv"], c["dk"], c["dv"]
    inside = s["inside"]
    chunks = _pad(inside.shape[1], CHUNK) // CHUNK

    def lay(x):
        full = torch.zeros(count, chunks * CHUNK, *x.shape[1:], device=DEV)
        full[:, :inside.shape[1]][inside] = x
        return full.unflatten(1, (chunks, CHUNK)).transpose(2, 3)

    q, k = (_unit(s[x], c["l2norm"]).repeat_interleave(hv // hk, 1) for x in ("q", "k"))
    q, k, v = lay(q * dk ** -0.5), lay(k), lay(s["v"].float())
    beta, g = lay(s["beta"])[..., None], torch.cumsum(lay(s["g"]).double(), 3)
    decay = torch.exp((g[..., :, None] - g[..., None, :]).tril()).tril().float()
    last = torch.exp(g[..., -1:] - g).float()[..., None]
    g = torch.exp(g).float()[..., None]
    lower = (k @ k.transpose(3, 4) * decay * beta).tril(-1)
    inverse = _unit_inverse(lower)
    u, w = inverse @ (v * beta), inverse @ (k * (g * beta))
    inner = q @ k.transpose(3, 4) * decay
    q, keys = q * g, (k * last).transpose(3, 4).contiguous()
    slots = s["slots"].long()
    state = torch.zeros(count, hv, dk, dv, device=DEV) if c["fresh"] else s["state"][slots]
    out = torch.empty(count, chunks, hv, CHUNK, dv, device=DEV)
    for i in range(chunks):
        new = u[:, i] - w[:, i] @ state
        out[:, i] = q[:, i] @ state + inner[:, i] @ new
        state = state * g[:, i, :, -1:] + keys[:, i] @ new
    s["state"][slots] = state
    s["out"].copy_(out.transpose(2, 3).flatten(1, 2)[:, :inside.shape[1]][inside])
    return {"out": s["out"], "state": s["state"]}


def _plain_recurrent(s):
    c = s["case"]
    count, tokens, hk, hv, dk = c["batch"], c["tokens"], c["hk"], c["hv"], c["dk"]
    q, k = (_unit(s[x], c["l2norm"]).repeat_interleave(hv // hk, 1).unflatten(0, (count, tokens)) for x in ("q", "k"))
    q, v = q * dk ** -0.5, s["v"].float().unflatten(0, (count, tokens))
    decay = torch.exp(s["g"]).view(count, tokens, hv, 1, 1)
    beta = s["beta"].view(count, tokens, hv, 1, 1)
    slots = s["slots"].long()
    state = s["state"][slots]
    out = torch.empty(count, tokens, hv, c["dv"], device=DEV)
    for i in range(tokens):
        state = state * decay[:, i]
        u = beta[:, i] * (v[:, i, :, None] - k[:, i, :, None] @ state)
        state = state + k[:, i, :, :, None] @ u
        out[:, i] = (q[:, i, :, None] @ state).squeeze(2)
    s["state"][slots] = state
    s["out"].copy_(out.flatten(0, 1))
    return {"out": s["out"], "state": s["state"]}


# ---- what one pass cannot do without --------------------------------------------------

def work(case):
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        out = {"bf16": 2 * m * k, "int8": m * k + 4 * m, "q8_1": m * _pad(k, 32) * 9 // 8}[case["out"]]
        return {"bytes": 2 * m * k + 2 * k + (4 * m * k if case["residual"] else 0) + out, "flops": 5 * m * k}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    if case["op"] == "chunked":
        lens, read = [int(n) for n in case["lens"].split()], 0 if case["fresh"] else 1
    else:
        lens, read = [case["tokens"]] * case["batch"], 1
    return {"bytes": sum(lens) * (4 * hk * dk + 4 * hv * dv + 8 * hv) + len(lens) * (read + 1) * 4 * hv * dk * dv,
            "flops": sum(lens) * hv * 6 * dk * dv}


# ---- the definitions, in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        h = x if s["residual"] is None else (x + s["residual"].double()).bfloat16().double()
        root = torch.sqrt((h * h).sum(1, keepdim=True) / case["k"] + EPS)
        n = h / root * s["weight"].double()
        if case["out"] == "int8":
            n = h * s["weight"].double()  # exact, so that the ties are: the root is common to a row
            top = n.abs().max(1, keepdim=True).values
            n = torch.round(127 * n / top) * (top / (127 * root))
        elif case["out"] == "q8_1":
            n = n.bfloat16().double()
            blocks = torch.nn.functional.pad(n, (0, -case["k"] % 32)).unflatten(1, (-1, 32))
            step = (blocks.abs().max(2, keepdim=True).values / 127).half().double()
            whole = torch.trunc(blocks.abs() / step + 0.5).clamp(max=127) * blocks.sign() * step
            n = whole.flatten(1)[:, :case["k"]]
        return {"y": n, "residual": None if s["residual"] is None else h}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = _split_int8_rows(s["act"], m, k)
        w, sw = _split_int8_rows(s["weight"], n, k)
        y = (a.double() * sa.double()[:, None]) @ (w.double() * sw.double()[:, None]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    # token by token, all sequences side by side; a sequence that has ended keeps its state
    hk, hv, dk = case["hk"], case["hv"], case["dk"]
    state, slots = s["state"].double(), s["slots"].long()
    S = state[slots]
    if case["op"] == "chunked" and case["fresh"]:
        S = torch.zeros_like(S)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["l2norm"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    q, k = (torch.repeat_interleave(x, hv // hk, dim=1) for x in (q / math.sqrt(dk), k))
    out = torch.zeros(v.shape, dtype=torch.float64, device=DEV)
    a, b = torch.exp(s["g"].double()), s["beta"].double()
    lens = torch.tensor(s["lens"])
    starts = s["starts"].long()
    for t in range(max(s["lens"])):
        live = None if int(lens.min()) > t else (lens > t).nonzero().flatten().to(DEV)
        at = starts[:-1] + t if live is None else starts[live] + t
        P = (S if live is None else S[live]) * a[at][:, :, None, None]
        kt = k[at][..., None]
        P = P + kt * (b[at][..., None] * (v[at] - (P * kt).sum(2)))[:, :, None]
        out[at] = (P * q[at][..., None]).sum(2)
        if live is None:
            S = P
        else:
            S[live] = P
    state[slots] = S
    return {"out": out, "state": state}
