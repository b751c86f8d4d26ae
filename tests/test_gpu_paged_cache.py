"""Rotary positions, head norms and the write of the paged cache, and its read-back, against the definition in 64 bits.

Bounds, with u = 2^-24: a rotated value is the sum of two products of at most three factors, each rounded, with the
norm's root and mean in binary32: off by (d + 16) u of the terms' magnitudes at most; then half a step of bf16, 2^-8, or
half a code, and a code is off by one where the quotient is next to a half: 0.5 + 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from paged_ref import Cache, Case, rope, table_of_angles

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = 2.0 ** -24


def make(lens, hq, hk, d, bits, page, seed, rot, axes=1, norm=False):
    """A case whose cache holds every byte 0xFF, and the packed rows of q, k and v."""
    c = Case([(n, total) for n, total in lens], hq, hk, d, bits, page, seed)
    c.cache = Cache(c.cache.pages, page, hk, d, bits)
    gen = torch.Generator().manual_seed(seed + 1)
    c.packed = torch.randn(c.tokens, (hq + 2 * hk) * d + 8, generator=gen).bfloat16()
    c.rot, c.axes = rot, axes
    c.cos_sin = table_of_angles(max((t for _, t in lens), default=1) + 4, rot)
    c.places = np.concatenate([np.arange(t - n, t) for n, t in lens] or [[]]).astype(np.int64)
    c.positions = c.axis = None
    if axes > 1:
        c.axis = (np.arange(rot // 2) % axes).astype(np.uint8)
        c.positions = np.stack([c.places // (a + 1) for a in range(axes)]).astype(np.int32)
    w = (1 + 0.2 * torch.randn(2, d, generator=gen)).bfloat16() if norm else None
    c.q_norm, c.k_norm = (None, None) if w is None else w
    return c


def split(c, packed):
    a, b = c.hq * c.d, c.hk * c.d
    return (packed[:, :a].unflatten(1, (c.hq, c.d)), packed[:, a:a + b].unflatten(1, (c.hk, c.d)),
            packed[:, a + b:a + 2 * b].unflatten(1, (c.hk, c.d)))


def write(c, gpu, t=None, **kw):
    t = c.device(gpu) if t is None else t
    q, k, v = split(c, c.packed.to(gpu))
    def dev(x):
        return None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(gpu)
    out = torch.full((c.tokens, c.hq, c.d), 7.0, dtype=torch.bfloat16, device=gpu)
    bq.rope_write_kv_cache(q, k, v, out, t["k_cache"], t["v_cache"], t["starts"], t["lens"], t["table"], c.page, c.bits,
                           cos_sin=dev(c.cos_sin) if c.rot else None, positions=dev(c.positions), axis=dev(c.axis),
                           q_norm=dev(c.q_norm), k_norm=dev(c.k_norm), eps=EPS, **kw)
    torch.cuda.synchronize()
    return out, t


def expected(c):
    rows = np.repeat(c.places[:, None], c.rot // 2, 1) if c.axis is None else c.positions[c.axis].T
    q, k, v = (x.double().numpy() for x in split(c, c.packed))
    cs = c.cos_sin.astype(np.float64)
    qn, kn = (None if w is None else w.double().numpy() for w in (c.q_norm, c.k_norm))
    return rope(q, cs, rows, qn, EPS), rope(k, cs, rows, kn, EPS), (v, np.abs(v))


def check_cache(c, t, keys, want, size):
    got = Cache(c.cache.pages, c.page, c.hk, c.d, c.bits)
    got.k, got.v = t["k_cache"].cpu().numpy().copy(), t["v_cache"].cpu().numpy().copy()
    seq = np.repeat(np.arange(len(c.lens)), [n for n, _ in c.lens])
    touched = np.zeros((c.cache.pages, c.page), dtype=bool)
    for i, p in enumerate(c.places):
        page_id = c.table[seq[i], p // c.page]
        touched[page_id, p % c.page] = True
        row = got.get(keys, page_id, p % c.page)
        err = (c.d + 16) * U * size[i] * (1 if keys else 0)
        if c.bits == 16:
            tol = 2.0 ** -8 * np.abs(want[i]) + 2 * err
        else:
            top = np.abs(want[i]).max(-1, keepdims=True)
            tol = (0.5 + 2.0 ** -10) * top / 127 + 2 * err + (c.d + 16) * U * top
        assert (np.abs(row - want[i]) <= tol).all(), (i, p)
    # the rest of the pool is as it was
    b = (got.k if keys else got.v).reshape(c.cache.pages, c.hk, c.cache.block)
    from paged_ref import places
    at = places(c.page, c.d, c.bits, keys)
    for page_id, o in zip(*np.nonzero(~touched)):
        if c.bits == 16:
            assert (b.view(np.uint16)[page_id][:, at[o]] == 0xFFFF).all()
        else:
            assert (b[page_id][:, at[o]] == 0xFF).all() and (b[page_id][:, c.page * c.d:].reshape(c.hk, c.page, 4)[:, o] == 0xFF).all()


SIZES = [
    # lens (new, all), hq, hk, d, page, rot, axes, norm
    ([(1, 1)], 1, 1, 16, 16, 16, 1, False),
    ([(1, 701)], 8, 2, 128, 64, 128, 1, False),
    ([(1, 38), (70, 70), (65, 100), (0, 5), (33, 49)], 4, 2, 256, 16, 64, 3, True),
    ([(5, 9), (40, 40)], 3, 1, 80, 32, 32, 1, True),
    ([(17, 17), (1, 16), (1, 17), (16, 32), (15, 31)], 6, 3, 96, 16, 96, 1, False),
    ([(20, 50)], 2, 2, 64, 1024, 0, 1, True),
    ([(9, 9)], 5, 5, 48, 16, 16, 2, False),
    ([(3, 3), (2, 130)], 40, 8, 192, 128, 192, 1, True),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_write_and_read(gpu, bits, size):
    lens, hq, hk, d, page, rot, axes, norm = SIZES[size]
    print(f"write bits={bits} {SIZES[size]}", flush=True)
    c = make(lens, hq, hk, d, bits, page, 40 + size, rot, axes, norm)
    out, t = write(c, gpu)
    (q, qs), (k, ks), (v, vs) = expected(c)
    assert (np.abs(out.double().cpu().numpy() - q) <= 2.0 ** -8 * np.abs(q) + 2 * (d + 16) * U * qs).all()
    check_cache(c, t, True, k, ks)
    check_cache(c, t, False, v, vs)
    # and back, what the bytes say rounded once
    kb, vb = (torch.full((c.tokens, hk, d), 7.0, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    bq.read_kv_cache(t["k_cache"], t["v_cache"], kb, vb, t["starts"], t["lens"], t["table"], page, bits)
    torch.cuda.synchronize()
    got = Cache(c.cache.pages, page, hk, d, bits)
    got.k, got.v = t["k_cache"].cpu().numpy(), t["v_cache"].cpu().numpy()
    seq = np.repeat(np.arange(len(lens)), [n for n, _ in lens])
    for keys, back in ((True, kb), (False, vb)):
        want = np.stack([got.get(keys, c.table[seq[i], p // page], p % page) for i, p in enumerate(c.places)])
        assert torch.equal(back.cpu(), torch.from_numpy(want).float().bfloat16())


def test_without_q(gpu):
    c = make([(5, 30)], 2, 2, 64, 16, 16, 50, 64)
    _, t = write(c, gpu)
    u = c.device(gpu)
    _, k, v = split(c, c.packed.to(gpu))
    bq.rope_write_kv_cache(None, k, v, None, u["k_cache"], u["v_cache"], u["starts"], u["lens"], u["table"], 16, 16,
                           cos_sin=torch.from_numpy(c.cos_sin).to(gpu))
    torch.cuda.synchronize()
    assert torch.equal(t["k_cache"], u["k_cache"]) and torch.equal(t["v_cache"], u["v_cache"])


def test_positions_that_are_no_rows_of_the_table(gpu):
    c = make([(4, 4)], 2, 1, 64, 16, 16, 51, 32)
    c.positions = np.array([0, 1 << 30, -1, 2], dtype=np.int32)
    out, t = write(c, gpu)
    out = out.float().cpu()
    assert out[[1, 2], :, :32].isnan().all() and out[:, :, 32:].isfinite().all() and out[[0, 3]].isfinite().all()
    c.positions, c.axis = np.zeros((2, 4), dtype=np.int32), np.full(16, 1, dtype=np.uint8)
    c.axis[3] = 2  # no such axis
    out, _ = write(c, gpu)
    assert out[:, :, [3, 19]].isnan().all() and out.isnan().sum() == 4 * 2 * 2


@pytest.mark.parametrize("bits", [16, 8])
def test_tokens_that_are_nowhere(gpu, bits):
    c = make([(6, 40), (3, 20)], 2, 1, 64, bits, 16, 52, 64)
    t = c.device(gpu)
    t["table"][0, 2] = -1              # places 32..39 of the first: nowhere
    t["lens"][1] = 2                   # its new tokens are at -1, 0, 1
    out, t = write(c, gpu, t)
    got = Cache(c.cache.pages, 16, 1, 64, bits)
    got.k, got.v = t["k_cache"].cpu().numpy(), t["v_cache"].cpu().numpy()
    page1 = c.table[1, 0]
    blocks = got.k.reshape(c.cache.pages, -1)
    others = [i for i in range(c.cache.pages) if i != page1]
    assert (blocks[others] == 0xFF).all() and (got.v.reshape(c.cache.pages, -1)[others] == 0xFF).all()
    assert np.isfinite(got.get(True, page1, 0)).all() and np.isfinite(got.get(False, page1, 1)).all()
    kb = torch.full((9, 1, 64), 7.0, dtype=torch.bfloat16, device=gpu)
    vb = kb.clone()
    bq.read_kv_cache(t["k_cache"], t["v_cache"], kb, vb, t["starts"], t["lens"], t["table"], 16, bits)
    torch.cuda.synchronize()
    assert (kb[:7] == 0).all() and (vb[:7] == 0).all() and kb[7:].isfinite().all() and (vb[7:] != 7).any()


def test_rows_that_int8_cannot_hold(gpu):
    c = make([(6, 6)], 1, 1, 64, 8, 16, 53, 0)
    rows = c.packed.float()
    rows[0, 64:128] = 0.0                       # k: zeros
    rows[1, 64 + 5] = float("nan")
    rows[2, 128 + 7] = float("inf")             # v
    rows[3, 64:128] *= 1e-38 / 128              # subnormal
    rows[4, 128:192] *= 5e37                    # near the largest
    c.packed = rows.bfloat16()
    _, t = write(c, gpu)
    got = Cache(c.cache.pages, 16, 1, 64, 8)
    got.k, got.v = t["k_cache"].cpu().numpy(), t["v_cache"].cpu().numpy()
    p = c.table[0, 0]
    assert (got.get(True, p, 0) == 0).all()
    assert np.isnan(got.get(True, p, 1)).all() and np.isnan(got.get(False, p, 2)).all()  # 0 * NaN, 0 * inf
    for keys, o, at in ((True, 3, 64), (False, 4, 128)):
        x = c.packed[o, at:at + 64].double().numpy()
        # (a scale below 2^-126 has fewer bits: 2^-150 off, 127 times)
        assert (np.abs(got.get(keys, p, o)[0] - x) <= 0.501 * np.abs(x).max() / 127 + 127 * 2.0 ** -149).all()


def test_replays_follow_the_lengths(gpu):
    c = make([(1, 40), (1, 18)], 2, 1, 64, 16, 16, 54, 64)
    t = c.device(gpu)
    q, k, v = split(c, c.packed.to(gpu))
    cs = torch.from_numpy(c.cos_sin).to(gpu)
    out = torch.empty(2, 2, 64, dtype=torch.bfloat16, device=gpu)

    def step(k_cache, v_cache):
        bq.rope_write_kv_cache(q, k, v, out, k_cache, v_cache, t["starts"], t["lens"], t["table"], 16, 16, cos_sin=cs)

    step(t["k_cache"], t["v_cache"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(t["k_cache"], t["v_cache"])
    for lens in ([40, 18], [33, 1], [16, 17]):
        t["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        t["k_cache"].fill_(0xFF)
        t["v_cache"].fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got, ko, vo = out.clone(), t["k_cache"].clone(), t["v_cache"].clone()
        k2, v2 = torch.full_like(ko, 0xFF), torch.full_like(vo, 0xFF)
        step(k2, v2)
        assert torch.equal(got, out) and torch.equal(ko, k2) and torch.equal(vo, v2)


@pytest.mark.parametrize("bits", [16, 8])
def test_prompt_then_tokens_through_the_cache(gpu, bits):
    """As they are used: a prompt is written and attended to, then tokens one by one; against one prompt of all."""
    n, more, hq, hk, d, page = 75, 5, 8, 2, 64, 16
    whole = make([(n + more, n + more)], hq, hk, d, bits, page, 60, d)
    t = whole.device(gpu)
    q, k, v = split(whole, whole.packed.to(gpu))
    cs = torch.from_numpy(whole.cos_sin).to(gpu)
    work = torch.empty(bq.paged_attention_workspace_bytes(n + more, 1, hq, hk, d), dtype=torch.uint8, device=gpu)

    def go(a, b, kc, vc, form):
        starts = torch.tensor([0, b - a], dtype=torch.int32, device=gpu)
        lens = torch.tensor([b], dtype=torch.int32, device=gpu)
        qo = torch.empty(b - a, hq, d, dtype=torch.bfloat16, device=gpu)
        out = torch.empty_like(qo)
        bq.rope_write_kv_cache(q[a:b], k[a:b], v[a:b], qo, kc, vc, starts, lens, t["table"], page, bits, cos_sin=cs)
        if form == "prefill":
            bq.paged_attention_prefill(qo, kc, vc, out, starts, lens, t["table"], hk, page, bits)
        else:
            bq.paged_attention_decode(qo, kc, vc, out, starts, lens, t["table"], work, hk, page, bits)
        return out

    parts = [go(0, n, t["k_cache"], t["v_cache"], "prefill")]
    parts += [go(n + i, n + i + 1, t["k_cache"], t["v_cache"], "decode") for i in range(more)]
    kc, vc = torch.full_like(t["k_cache"], 0xFF), torch.full_like(t["v_cache"], 0xFF)
    all_at_once = go(0, n + more, kc, vc, "prefill")
    torch.cuda.synchronize()
    assert torch.equal(kc, t["k_cache"]) and torch.equal(vc, t["v_cache"])
    one, two = torch.cat(parts).double(), all_at_once.double()
    assert (one - two).norm() <= 3 * 2.0 ** -8 * two.norm()
