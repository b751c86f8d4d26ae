"""The paged cache and the attention over it at the ends of their arguments' and values' ranges: values that are not
finite, in tiles that all rows see and in tiles that some see; the largest values; scales and caps; ties between int8
codes (bounds: paged_ref.bound)."""
import numpy as np
import pytest
import torch

from paged_ref import Cache, Case, attention, bound
from test_gpu_paged_attention import FORMS, call, check
from test_gpu_paged_cache import make, write
from test_gpu_paged_variants import widened

pytestmark = pytest.mark.gpu


def planted(case, seq, marks):
    """The case's cache with these (place, column, value) in the values of a sequence, in all heads."""
    for place in sorted({p for p, _, _ in marks}):
        v = case.rows[seq][1][place].copy()
        for p, column, value in marks:
            if p == place:
                v[:, column] = value
        case.cache.put(False, case.table[seq, place // case.page], place % case.page, v)


def check_planted(case, out, clean, seq, marks, window=0):
    """What was planted reaches the rows that see it, in its column, and all else is as without: the same sums in another
    order in binary32, and half a step of bf16 for each of the two."""
    out, clean = out.float().cpu(), clean.float().cpu()
    n, total = case.lens[seq]
    for i in range(n):
        pos, row = total - n + i, int(case.starts[seq]) + i
        for column in {c for _, c, _ in marks}:
            seen = [v for p, c, v in marks if c == column and p <= pos and (not window or p > pos - window)]
            if seen:
                want = torch.tensor(float(sum(seen)))  # inf - inf is a NaN
                got = out[row, :, column]
                assert (got.isnan() if want.isnan() else got == want).all(), (row, column, got)
                out[row, :, column] = clean[row, :, column]
    assert ((out - clean).abs() <= 2.0 ** -7 * clean.abs() + 2.0 ** -14).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("hole", [None, 64])
@pytest.mark.parametrize("d,page", [(64, 64), (128, 64), (256, 64), (128, 16), (80, 32)])
def test_nan_in_tiles_that_all_rows_see(gpu, form, window, hole, d, page):
    # few workgroups: two groups of waves take the tiles of keys in turn, and one's tile may be seen whole, the other's not
    print(f"nan {form} window={window} hole={hole} d={d} page={page}", flush=True)
    case = Case([(256, 256)], 8, 2, d, 16, page, 800 + d)
    if hole is not None:
        case.table[0, hole // page] = -1
    clean = call(form, case, case.device(gpu), window=window)
    marks = [(10, 1, np.nan), (45, 2, np.nan), (130, 3, np.nan), (150, 4, np.nan), (200, 5, np.nan)]
    planted(case, 0, marks)
    out = call(form, case, case.device(gpu), window=window)
    torch.cuda.synchronize()
    check_planted(case, out, clean, 0, marks, window)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("scale,window,cap", [(0.0, 0, 0.0), (0.0, 50, 0.0), (0.0, 0, 3.0), (1e-45, 50, 0.0), (1e-30, 0, 0.0), (0.4, 50, 0.0), (0.4, 0, 3.0)])
def test_scales(gpu, form, bits, scale, window, cap):
    # scale 0: the mean of the values that are seen
    print(f"scale {form} bits={bits} scale={scale} window={window} cap={cap}", flush=True)
    for case in (Case([(3, 400), (1, 5), (20, 20), (2, 130)], 6, 2, 64, bits, 16, 900),
                 widened(Case([(1, 1500), (7, 300), (2, 129)], 4, 1, 128, bits, 32, 901))):
        out = call(form, case, case.device(gpu), window=window, cap=cap, scale=scale)
        torch.cuda.synchronize()
        check(form, case, out, window=window, cap=cap, scale=scale)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("cap,spread", [(50.0, 1.0), (64.0, 40.0), (65.0, 40.0), (100.0, 60.0), (1e3, 1.0), (1e3, 300.0), (1e5, 1.0), (1e6, 4.0),
                                        (1e8, 1.0), (1e20, 1.0)])
def test_caps(gpu, form, bits, page, cap, spread):
    # the bound has no term that grows with the cap: caps that are far above the scores leave them as they are
    print(f"cap {form} bits={bits} page={page} cap={cap} spread={spread}", flush=True)
    for case in (Case([(3, 400), (1, 5), (20, 20), (2, 130)], 6, 2, 64, bits, page, 910, spread=spread),
                 widened(Case([(1, 1500), (9, 300), (2, 129)], 4, 1, 128, bits, page, 911, spread=spread))):
        out = call(form, case, case.device(gpu), cap=cap)
        torch.cuda.synchronize()
        ref, size, most = attention(case, cap=cap)
        off = np.abs(out.double().cpu().numpy() - ref)
        far = off - bound(case, ref, size, most, form)
        assert np.isfinite(off).all() and far.max() <= 0, f"off by {off.max():.3e}, {far.max():.3e} over the bound"


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_caps_far_below_the_scores(gpu, form, bits):
    # scale / cap is beyond binary32; a query of zeros, whose scores are 0
    case = Case([(3, 400), (20, 20)], 6, 2, 64, bits, 16, 912)
    case.packed[1] = 0
    out = call(form, case, case.device(gpu), cap=1e-20, scale=1e30)
    torch.cuda.synchronize()
    check(form, case, out, cap=1e-20, scale=1e30)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("keys", [0, 4096])
@pytest.mark.parametrize("d,hq", [(64, 4), (64, 16), (80, 4), (128, 4), (128, 16), (256, 4), (256, 16)])
def test_infinities(gpu, form, keys, d, hq):
    # each in a column of its own, in steps that all rows see and in steps that some see; and two that make a NaN
    print(f"inf {form} keys={keys} d={d} hq={hq}", flush=True)
    case = widened(Case([(20, 700), (1, 900), (9, 60)], hq, 2, d, 16, 64, 920 + d), keys)
    clean = call(form, case, case.device(gpu))
    inf = np.inf
    marks = [[(3, 1, inf), (40, 2, -inf), (100, 3, inf), (333, 4, inf), (685, 5, -inf), (695, 6, inf), (50, 7, inf), (690, 7, -inf)],
             [(0, 1, -inf), (31, 2, inf), (500, 3, inf), (899, 4, -inf)], [(54, 8, inf), (10, 9, -inf)]]
    for seq, m in enumerate(marks):
        planted(case, seq, m)
    out = call(form, case, case.device(gpu))
    torch.cuda.synchronize()
    for seq, m in enumerate(marks):
        rows = slice(int(case.starts[seq]), int(case.starts[seq + 1]))
        one = Case.__new__(Case)
        one.lens, one.starts = [case.lens[seq]], np.array([0, case.lens[seq][0]])
        check_planted(one, out[rows], clean[rows], 0, m)


def test_codes_are_the_nearest(gpu):
    # rows of all magnitudes; with halves of the largest value, whose quotients lie between two codes
    n, hk, d = 400, 2, 64
    c = make([(n, n)], 1, hk, d, 8, 16, 930, 0)
    gen = torch.Generator().manual_seed(931)
    top = torch.rand(n, 2 * hk, 1, generator=gen) + 1
    x = torch.rand(n, 2 * hk, d, generator=gen) * 2 - 1
    x[..., 0], x[..., 1], x[..., 2] = 1, 0.5, -0.5
    power = torch.randint(-133, 127, (n, 2 * hk, 1), generator=gen).double()
    x = (x.double() * (top.bfloat16().double() * torch.exp2(power)))
    c.packed[:, d:d + 2 * hk * d] = x.bfloat16().flatten(1)
    _, t = write(c, gpu)
    got = Cache(c.cache.pages, 16, hk, d, 8)
    got.k, got.v = t["k_cache"].cpu().numpy(), t["v_cache"].cpu().numpy()
    x = c.packed[:, d:d + 2 * hk * d].float().numpy().reshape(n, 2 * hk, d)
    for keys in (True, False):
        rows = x[:, :hk] if keys else x[:, hk:]
        for p in range(n):
            for h in range(hk):
                block, at = got._at(keys, c.table[0, p // 16], h)
                big = np.abs(rows[p, h]).max()
                scaled = rows[p, h].astype(np.float64) * 127  # exact; so is the nearest code of the quotient in 64 bits
                want = np.rint(scaled / big) if big else np.zeros(d)
                assert (block[:16 * d].view(np.int8)[at[p % 16]] == want).all(), (keys, p, h)
                assert block[16 * d:].view(np.float32)[p % 16] == big / np.float32(127)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d,keys", [(64, 0), (64, 4096), (128, 0), (128, 4096), (256, 4096)])
def test_large_values(gpu, form, bits, d, keys):
    # values whose sum is just below 2^128, behind keys with lower scores (by a factor of 2^7.5 in the weights), so that
    # the running maximum is one of those
    n, low = (2000, 1152) if keys else (960, 512)
    case = Case([(1, n), (40, n)], 2, 1, d, bits, 64, 940)
    case.packed.zero_()
    case.packed[:, 0:2 * d:d] = 1
    for seq in range(2):
        for p in range(n):
            k, v = np.zeros((1, d)), np.full((1, d), 2.0 ** 116)
            k[0, 0] = 0.0 if p < low else 5.1875
            for rows, keyed in ((k, True), (v, False)):
                case.rows[seq][0 if keyed else 1][p] = rows
                if bits == 8:
                    top = np.abs(rows).max()
                    scale = np.float32(top / 127)
                    rows = (np.rint(rows / (top or 1) * 127).astype(np.int8), np.full(1, scale, dtype=np.float32))
                    case.rows[seq][0 if keyed else 1][p] = rows[0] * rows[1].astype(np.float64)[:, None]
                case.cache.put(keyed, case.table[seq, p // 64], p % 64, rows)
    if keys:
        case = widened(case, keys)
    out = call(form, case, case.device(gpu), scale=1.0)
    torch.cuda.synchronize()
    check(form, case, out, scale=1.0)
