"""The paged cache and the attention over it at the ends of their arguments' and values' ranges: values that are not
finite, in tiles that all rows see and in tiles that some see; scales (bounds: paged_ref.bound)."""
import numpy as np
import pytest
import torch

from paged_ref import Case
from test_gpu_paged_attention import FORMS, call, check
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
