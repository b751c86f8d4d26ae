"""Attention over the paged cache where the launch chooses between kernels: long tables (sequences cut into runs and
joined), many workgroups (one group of waves to a tile of rows), all head sizes and types of both; pools beyond 4 GiB,
two streams at once, one workspace under two graphs (bounds: paged_ref.bound)."""
import numpy as np
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from paged_ref import Case, attention
from test_gpu_paged_attention import FORMS, call, check

pytestmark = pytest.mark.gpu
HEADS = [16, 64, 80, 96, 128, 192, 256]


def widened(case, keys=4096):
    """The table with room for more than `keys` keys, the entries behind the sequences' pages nowhere."""
    width = max(case.table.shape[1], keys // case.page + 1)
    table = np.full((len(case.lens), width), -1, dtype=np.int32)
    table[:, :case.table.shape[1] - 1] = case.table[:, :-1]
    case.table = table
    return case


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d", HEADS)
def test_cut_sequences(gpu, d, bits, rows, page):
    # few: up to 16 rows a key head on average; many: above.  Runs that begin and end inside sequences, and sequences
    # that end within a block of keys
    lens = [(1, 1500), (2, 65), (0, 30), (1, 1), (3, 700)] if rows == "few" else [(9, 1100), (5, 130), (12, 12), (1, 320)]
    print(f"cut d={d} bits={bits} {rows} page={page}", flush=True)
    case = widened(Case(lens, 8, 2, d, bits, page, 200 + d))
    out = call("decode", case, case.device(gpu))
    torch.cuda.synchronize()
    check("decode", case, out)


@pytest.mark.parametrize("d,bits,window,cap", [(64, 16, 100, 0.0), (128, 8, 33, 0.0), (128, 16, 0, 3.0), (256, 8, 500, 4.0), (80, 16, 1, 0.0),
                                               (256, 16, 64, 0.0)])
def test_cut_sequences_under_windows_and_caps(gpu, d, bits, window, cap):
    print(f"cut d={d} bits={bits} window={window} cap={cap}", flush=True)
    case = widened(Case([(1, 1500), (7, 300), (30, 30), (2, 129)], 4, 1, d, bits, 32, 300 + d, spread=2.0))
    out = call("decode", case, case.device(gpu), window=window, cap=cap)
    torch.cuda.synchronize()
    check("decode", case, out, window=window, cap=cap)


@pytest.mark.parametrize("d,hq", [(64, 4), (64, 16), (128, 4), (256, 16), (80, 4)])
def test_nan_in_cut_sequences(gpu, d, hq):
    # a NaN in the values of one token and an infinity in a later one's: the rows before them as without, those that
    # see them NaN in that column
    case = widened(Case([(20, 700), (1, 900)], hq, 2, d, 16, 64, 400 + d))
    t = case.device(gpu)
    clean = call("decode", case, t).float().cpu()
    for place, what in ((685, np.nan), (695, -np.inf)):
        v = case.rows[0][1][place].copy()
        v[:, 3] = what
        case.cache.put(False, case.table[0, place // 64], place % 64, v)
    out = call("decode", case, case.device(gpu)).float().cpu()
    sees = torch.zeros(21, dtype=torch.bool)
    sees[5:20] = True  # token i is at place 680 + i
    assert out[sees][:, :, 3].isnan().all()
    out[sees.nonzero()[:, 0], :, 3] = clean[sees][:, :, 3]
    assert ((out - clean).abs() <= 2.0 ** -7 * clean.abs() + 2.0 ** -14).all()


def test_rows_of_no_sequence_beside_cut_ones(gpu):
    # rows before the first and behind the last sequence stay as they were, whatever the workspace holds
    case = widened(Case([(2, 900), (3, 1300)], 4, 2, 64, 16, 64, 450))
    t = case.device(gpu)
    whole = call("decode", case, t)
    t["starts"] = torch.tensor([0, 2, 4], dtype=torch.int32, device=gpu)  # the second's last two of 1299 tokens
    t["lens"] = torch.tensor([900, 1299], dtype=torch.int32, device=gpu)
    for fill in (0x00, 0x01, 0xFF):
        work = torch.full((bq.paged_attention_workspace_bytes(5, 2, 4, 2, 64),), fill, dtype=torch.uint8, device=gpu)
        out = call("decode", case, t, None, work)
        assert (out[4] == 7).all() and ((out[:4] - whole[:4]).abs() <= 2.0 ** -7 * whole[:4].abs() + 2.0 ** -14).all()


# 65 sequences and more of 8 key heads: more than 512 workgroups of 128 rows
MANY = [(1 + i % 3, 1 + (i * 29) % 60 + 3) for i in range(68)] + [(150, 150), (130, 300)]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d", HEADS)
def test_many_workgroups(gpu, d, bits, page):
    print(f"many workgroups d={d} bits={bits} page={page}", flush=True)
    case = Case(MANY, 8, 8, d, bits, page, 500 + d)
    out = call("prefill", case, case.device(gpu))
    torch.cuda.synchronize()
    check("prefill", case, out)


@pytest.mark.parametrize("hk,d,bits,window,cap", [(10, 64, 16, 40, 0.0), (10, 128, 8, 100, 0.0), (10, 128, 16, 0, 2.0), (10, 256, 8, 17, 3.0),
                                                  (10, 80, 8, 64, 5.0), (10, 96, 16, 130, 0.0), (10, 256, 16, 31, 2.0)])
def test_many_workgroups_under_windows_and_caps(gpu, hk, d, bits, window, cap):
    # up to 64 sequences: those with the most keys first
    print(f"many workgroups hk={hk} d={d} bits={bits} window={window} cap={cap}", flush=True)
    case = Case([(i % 3, 3 + (i * 29) % 60) for i in range(62)] + [(150, 150), (130, 300)], hk, hk, d, bits, 64, 600 + d, spread=2.0)
    out = call("prefill", case, case.device(gpu), window=window, cap=cap)
    torch.cuda.synchronize()
    check("prefill", case, out, window=window, cap=cap)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_among_many_workgroups(gpu, d, bits):
    # a value that is not finite (a scale, in int8) within a tile that some rows see in part
    case = Case(MANY, 8, 8, d, bits, 64, 700 + d)
    clean = call("prefill", case, case.device(gpu)).float().cpu()
    if bits == 16:
        v = case.rows[68][1][75].copy()
        v[:, 3] = np.nan
    else:
        v = np.zeros((8, d), dtype=np.int8), np.full(8, np.inf, dtype=np.float32)
    case.cache.put(False, case.table[68, 75 // 64], 75 % 64, v)
    out = call("prefill", case, case.device(gpu)).float().cpu()
    sees = torch.zeros(case.tokens, dtype=torch.bool)
    sees[int(case.starts[68]) + 75:int(case.starts[69])] = True
    if bits == 16:
        assert out[sees][:, :, 3].isnan().all()
        out[sees.nonzero()[:, 0], :, 3] = clean[sees][:, :, 3]
    else:
        assert out[sees].isnan().all()
        out[sees] = clean[sees]
    assert ((out - clean).abs() <= 2.0 ** -7 * clean.abs() + 2.0 ** -14).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits", [16, 8])
def test_pages_beyond_4_gib(gpu, form, bits):
    # the same pages at the end of a pool of 5 GiB, under as much larger numbers
    case = Case([(3, 200), (1, 70)], 8, 2, 128, bits, 64, 21)
    t = case.device(gpu)
    want = call(form, case, t)
    page_bytes = case.cache.block * 2
    pages = 5 * 2 ** 30 // page_bytes
    ahead = pages - case.cache.pages
    for name in ("k_cache", "v_cache"):
        large = torch.empty(pages * page_bytes, dtype=torch.uint8, device=gpu)
        large[ahead * page_bytes:] = t[name]
        t[name] = large
    t["table"] = torch.where((t["table"] >= 0) & (t["table"] < case.cache.pages), t["table"] + ahead, t["table"])
    assert torch.equal(call(form, case, t), want)


@pytest.mark.parametrize("keys", [0, 4096])
def test_two_streams_at_once(gpu, keys):
    # a workspace each; many calls of different sequences that overlap
    cases = [Case([(1, 900), (2, 60)], 8, 2, 128, 16, 64, 22), Case([(1, 500), (1, 33), (4, 800)], 8, 2, 128, 16, 64, 23)]
    if keys:
        cases = [widened(c, keys) for c in cases]
    ts = [c.device(gpu) for c in cases]
    want = [call("decode", c, t) for c, t in zip(cases, ts)]
    works = [torch.full((bq.paged_attention_workspace_bytes(c.tokens, len(c.lens), 8, 2, 128),), 0xFF, dtype=torch.uint8, device=gpu) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for c, t, work, s, out in zip(cases, ts, works, streams, outs):
            with torch.cuda.stream(s):
                call("decode", c, t, out[i], work)
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        assert all(torch.equal(o, w) for o in out)


def test_one_workspace_under_two_graphs(gpu):
    # replayed in turn on one stream, also with a call between them that leaves other runs in the workspace
    cases = [widened(Case([(1, 900), (2, 60)], 8, 2, 128, 16, 64, 24)), widened(Case([(3, 1300)], 8, 2, 128, 16, 64, 25))]
    ts = [c.device(gpu) for c in cases]
    work = torch.full((max(bq.paged_attention_workspace_bytes(c.tokens, len(c.lens), 8, 2, 128) for c in cases),), 0xFF, dtype=torch.uint8, device=gpu)
    want = [call("decode", c, t) for c, t in zip(cases, ts)]
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for c, t, out in zip(cases, ts, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call("decode", c, t, out, work)
        graphs.append(graph)
    for turn in range(6):
        for out, w, graph in zip(outs, want, graphs):
            out.zero_()
            graph.replay()
            if turn % 2:
                call("decode", cases[0], ts[0], None, work)
            torch.cuda.synchronize()
            assert torch.equal(out, w)


def test_calls_repeat_their_results(gpu):
    # nothing depends on the order in which workgroups end
    case = widened(Case([(9, 1100), (5, 130), (12, 12), (1, 320)], 8, 2, 128, 8, 64, 26))
    t = case.device(gpu)
    for form in FORMS:
        want = call(form, case, t)
        assert all(torch.equal(call(form, case, t), want) for _ in range(5))
