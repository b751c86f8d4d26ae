"""Attention over the paged cache, both forms, against the definition in 64 bits (bounds: paged_ref.bound).

The cache holds NaN in every place that no token has: the rest of pages, and pages of nobody; entries of the table
behind a sequence's end are outside the pool."""
import numpy as np
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from paged_ref import Case, attention, bound

pytestmark = pytest.mark.gpu
FORMS = ["decode", "prefill"]


def call(form, case, t, out=None, work=None, **kw):
    out = torch.full((case.tokens, case.hq, case.d), 7.0, dtype=torch.bfloat16, device=t["k_cache"].device) if out is None else out
    args = (t["q"], t["k_cache"], t["v_cache"], out, t["starts"], t["lens"], t["table"])
    if form == "decode":
        size = bq.paged_attention_workspace_bytes(case.tokens, len(case.lens), case.hq, case.hk, case.d)
        if work is None:
            work = torch.full((size,), 0xFF, dtype=torch.uint8, device=out.device)  # NaN wherever it is read unwritten
        bq.paged_attention_decode(*args, work, case.hk, case.page, case.bits, **kw)
    else:
        bq.paged_attention_prefill(*args, case.hk, case.page, case.bits, **kw)
    return out


def check(form, case, out, **kw):
    ref, size, most = attention(case, **kw)
    off = np.abs(out.double().cpu().numpy() - ref)
    far = off - bound(case, ref, size, most, form, kw.get("cap", 0.0))
    assert np.isfinite(off).all() and far.max() <= 0, f"off by {off.max():.3e}, {far.max():.3e} over the bound at {np.unravel_index(far.argmax(), far.shape)}"


SIZES = [
    # lens (new, all), hq, hk, d, page
    ([(1, 1)], 1, 1, 16, 16),
    ([(1, 1), (2, 2), (3, 5)], 4, 2, 64, 16),
    ([(1, 700)], 8, 2, 128, 64),
    ([(1, 64), (1, 65), (1, 63), (1, 1), (1, 300)], 8, 2, 128, 32),
    ([(4, 130), (1, 17), (0, 40), (8, 8)], 12, 3, 80, 16),
    ([(4, 500), (4, 33)], 16, 2, 256, 128),
    ([(2, 300)], 24, 1, 96, 16),
    ([(5, 90), (3, 200)], 6, 6, 48, 64),
    ([(1, 257), (1, 1000)], 40, 2, 192, 32),
    ([(70, 70), (1, 33), (33, 161)], 4, 1, 64, 16),
    ([(129, 200)], 2, 2, 128, 64),
    ([(150, 150)], 3, 1, 256, 64),
    ([(40, 300)], 8, 2, 192, 16),
    ([(65, 129)], 5, 1, 32, 1024),
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_attention(gpu, form, bits, size):
    lens, hq, hk, d, page = SIZES[size]
    print(f"attention {form} bits={bits} {SIZES[size]}", flush=True)
    case = Case(lens, hq, hk, d, bits, page, 100 + size)
    out = call(form, case, case.device(gpu))
    torch.cuda.synchronize()
    check(form, case, out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("window,cap,spread", [(1, 0.0, 1.0), (7, 0.0, 1.0), (64, 0.0, 3.0), (100, 5.0, 4.0), (0, 2.0, 3.0), (1000, 0.0, 1.0)])
def test_windows_and_caps(gpu, form, bits, window, cap, spread):
    print(f"window {form} bits={bits} window={window} cap={cap}", flush=True)
    case = Case([(3, 400), (1, 5), (20, 20), (2, 130)], 6, 2, 64, bits, 16, 7, spread=spread)
    out = call(form, case, case.device(gpu), window=window, cap=cap)
    torch.cuda.synchronize()
    check(form, case, out, window=window, cap=cap)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_scores_far_apart(gpu, form, bits):
    # a row's scores span hundreds: the running maximum moves by more than its slack, up and down the keys
    case = Case([(2, 700), (50, 300)], 4, 2, 128, bits, 64, 11, spread=30.0)
    out = call(form, case, case.device(gpu))
    torch.cuda.synchronize()
    check(form, case, out)


@pytest.mark.parametrize("bits", [16, 8])
def test_long_sequences_are_cut(gpu, bits):
    # lengths that differ by thousands, so that runs of all lengths and joins occur
    case = Case([(1, 9000), (1, 3), (2, 4097), (1, 0 + 513)], 4, 1, 64, bits, 64, 12)
    t = case.device(gpu)
    out = call("decode", case, t)
    torch.cuda.synchronize()
    check("decode", case, out)
    again = call("decode", case, t)
    assert torch.equal(out, again)


@pytest.mark.parametrize("form", FORMS)
def test_nan_stays_with_the_tokens_that_see_it(gpu, form):
    # an infinity and a NaN in values of later tokens, and a NaN in a key: earlier tokens are as before
    case = Case([(40, 100)], 4, 2, 64, 16, 16, 13)
    case_clean = Case([(40, 100)], 4, 2, 64, 16, 16, 13)
    clean = call(form, case, case.device(gpu))
    for place, what in ((75, "v"), (99, "v"), (90, "k")):
        rows = case.rows[0][0 if what == "k" else 1][place].copy()
        rows[:, 5] = np.nan if place != 99 else np.inf
        case.cache.put(what == "k", case.table[0, place // 16], place % 16, rows)
    out = call(form, case, case.device(gpu))
    torch.cuda.synchronize()
    out, clean = out.float().cpu(), clean.float().cpu()
    # token i is at place 60 + i: 15 sees the NaN value, 30 the NaN key, 39 the infinity.  Sums in another order:
    # in binary32, then half a step of bf16 each
    near = (out - clean).abs() <= 2.0 ** -7 * clean.abs() + 2.0 ** -16 * attention(case_clean)[1].max()
    assert near[:15].all() and near[15:30, :, :5].all() and near[15:30, :, 6:].all()
    assert out[15:, :, 5].isnan().all() and out[30:].isnan().all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hq,hk,page,window", [(4, 2, 16, 0), (2, 2, 64, 30), (16, 1, 32, 0)])
def test_nan_scales_stay_with_the_tokens_that_see_them(gpu, form, hq, hk, page, window):
    # int8 rows that held a NaN: zero codes, and the NaN as their scale; of a value, and of a key
    case = Case([(40, 100), (200, 200)], hq, hk, 64, 8, page, 20)
    clean = call(form, case, case.device(gpu), window=window)
    for seq, place, keys in ((0, 75, False), (0, 90, True), (1, 130, False)):
        codes, scales = np.zeros((hk, 64), dtype=np.int8), np.full(hk, np.nan, dtype=np.float32)
        case.cache.put(keys, case.table[seq, place // page], place % page, (codes, scales))
    out = call(form, case, case.device(gpu), window=window)
    torch.cuda.synchronize()
    near = (out.float() - clean.float()).abs() <= 2.0 ** -6 * clean.float().abs() + 2.0 ** -9
    reach = window or 1 << 30
    sees = torch.zeros(240, dtype=torch.bool)
    for row in range(240):
        seq, pos = (0, 60 + row) if row < 40 else (1, row - 40)
        sees[row] = any(s == seq and p <= pos < p + reach for s, p in ((0, 75), (0, 90), (1, 130)))
    assert out[sees.to(gpu)].isnan().all() and near[~sees.to(gpu)].all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_places_that_are_nowhere(gpu, form, bits):
    # a page in the middle that is outside the pool, tokens before the beginning, lengths beyond the table
    case = Case([(3, 200), (2, 40), (1, 30)], 4, 2, 64, bits, 16, 14)
    t = case.device(gpu)
    t["table"][0, 5] = -1
    t["lens"][1] = 1     # its two new tokens are at places -1 and 0
    t["lens"][2] = 1 << 30
    out = call(form, case, t)
    torch.cuda.synchronize()
    ks, vs = case.rows[0]
    keep = np.r_[0:80, 96:200]
    q = case.q()
    for tok in range(3):
        for h in range(4):
            sel = keep[keep <= 197 + tok]
            s = 64 ** -0.5 * (ks[sel, h // 2] @ q[tok, h])
            w = np.exp(s - s.max())
            ref = w @ vs[sel, h // 2] / w.sum()
            assert np.abs(out[tok, h].double().cpu().numpy() - ref).max() <= 2.0 ** -7 * (w @ np.abs(vs[sel, h // 2]) / w.sum()).max()
    assert (out[3] == 0).all()  # before the beginning: nothing is seen
    one = np.repeat(case.rows[1][1][0], 2, 0)  # one key: its value, the weight and the output rounded
    assert (np.abs(out[4].double().cpu().numpy() - one) <= 2.0 ** -7 * np.abs(one) * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("form", FORMS)
def test_rows_of_no_sequence_are_left(gpu, form):
    case = Case([(2, 40), (3, 50)], 4, 2, 64, 16, 16, 15)
    t = case.device(gpu)
    t["starts"] = torch.tensor([0, 2, 4], dtype=torch.int32, device=gpu)  # the last row is nobody's
    out = call(form, case, t)
    torch.cuda.synchronize()
    assert (out[4] == 7).all() and not (out[:4] == 7).any()
    t["starts"] = torch.tensor([1, 2, 90], dtype=torch.int32, device=gpu)  # cut off at the last row
    out = call(form, case, t)
    torch.cuda.synchronize()
    assert (out[0] == 7).all()


@pytest.mark.parametrize("form", FORMS)
def test_many_sequences(gpu, form):
    # more than a wave's lanes, some without tokens
    lens = [((i * 7) % 3, 1 + (i * 37) % 90) for i in range(150)]
    case = Case([(min(n, total), total) for n, total in lens], 2, 1, 32, 16, 16, 16)
    out = call(form, case, case.device(gpu))
    torch.cuda.synchronize()
    check(form, case, out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_replays_read_lengths_anew(gpu, form, bits):
    # captured once, replayed as the sequences grow and other pages are taken, other work between the replays
    case = Case([(2, 300), (1, 77)], 4, 2, 64, bits, 16, 17)
    t = case.device(gpu)
    work = torch.full((bq.paged_attention_workspace_bytes(3, 2, 4, 2, 64),), 0xFF, dtype=torch.uint8, device=gpu)
    out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device=gpu)
    call(form, case, t, out, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(form, case, t, out, work)
    for lens in ([300, 77], [20, 3], [299, 60], [2, 1]):
        t["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        work.fill_(0xFF)
        want = call(form, case, t, None, work)
        assert torch.equal(got, want)


@pytest.mark.parametrize("form", FORMS)
def test_on_another_stream_with_one_head(gpu, form):
    # strides that one token and one head do not use are any; a stream of its own
    case = Case([(1, 50)], 1, 1, 64, 16, 16, 18)
    t = case.device(gpu)
    t["q"] = t["q"].as_strided((1, 1, 64), (3, 5, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = call(form, case, t)
    side.synchronize()
    check(form, case, out)


def test_forms_agree(gpu):
    case = Case([(64, 700), (64, 64)], 8, 2, 128, 16, 64, 19)
    t = case.device(gpu)
    one, two = call("decode", case, t).double(), call("prefill", case, t).double()
    # two outputs rounded to bf16, and weights rounded to bf16 in one: three times 2^-8 of what is summed
    assert (one - two).norm() <= 3 * 2.0 ** -8 * two.norm()
