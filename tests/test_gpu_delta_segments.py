"""Long sequences of few heads, which the chunked gated delta rule cuts into segments that run side by side: the same
definition and bounds as in test_gpu_delta_rule (a segment's state is a product of fewer roundings than the chain's:
one per segment where the chain has them per token)."""
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from test_gpu_delta_rule import call, check, heads, make

pytestmark = pytest.mark.gpu


def is_cut(tokens, count, hk, hv, dk, dv):
    """Whether these sizes need more than what a head needs where there are heads enough."""
    size = bq.gated_delta_rule_workspace_bytes
    return 64 * size(tokens, count, hk, hv, dk, dv) > size(tokens, count, 64 * hk, 64 * hv, dk, dv)


SIZES = [(1, 1, 128, 128), (1, 2, 64, 64), (1, 1, 128, 80), (2, 2, 100, 7), (1, 1, 33, 40), (1, 1, 65, 130), (1, 1, 1, 1)]
LENS = [[2048], [2177], [3100, 0, 3, 5700], [64 * 40, 64 * 41 + 1], [5, 5000]]


@pytest.mark.parametrize("lens", LENS, ids=lambda l: "-".join(map(str, l)))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_definition(gpu, sizes, lens):
    print(f"delta segments {sizes} {lens}", flush=True)
    assert is_cut(sum(lens), len(lens), *sizes)
    l2norm = (len(lens) + sizes[3]) % 3 != 0
    d = make(lens, *sizes, seed=sum(lens) + sum(sizes), l2norm=l2norm)
    fresh = [(i + 1) % 2 for i in range(len(lens))]
    check(d, *call(gpu, "chunked", d, fresh), fresh)


def test_state_carries_through_every_segment(gpu):
    """No decay, small betas: the first state is still there at the end, and goes through every product."""
    d = make([2500], 1, 1, 128, 64, seed=21)
    assert is_cut(2500, 1, 1, 1, 128, 64)
    d["g"].zero_()
    d["beta"] *= 1e-3
    d["state"] *= 100
    check(d, *call(gpu, "chunked", d))


def test_strong_decay_and_forgetting(gpu):
    d = make([2000], 1, 2, 64, 48, seed=22, strong=True)
    assert is_cut(2000, 1, 1, 2, 64, 48)
    d["g"][640, 0] = d["g"][1999, 1] = d["g"][128, 1] = float("-inf")
    out, state = call(gpu, "chunked", d)
    assert out.isfinite().all() and state.isfinite().all()
    check(d, out, state)


def test_slots_outside_and_ranges_cut_off(gpu):
    d = make([2500, 2100], 1, 1, 64, 32, seed=23, slots=None)
    assert is_cut(4600, 2, 1, 1, 64, 32)
    d["slots"] = torch.tensor([-1, 4], dtype=torch.int32)  # four slots: 0..3
    check(d, *call(gpu, "chunked", d))
    d["slots"] = torch.tensor([2, 0], dtype=torch.int32)
    want = call(gpu, "chunked", d)
    check(d, *want)
    d["starts"] = [-70, 2500, 9000]
    got = call(gpu, "chunked", d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_nothing_reads_a_fresh_slot_or_a_foreign_token(gpu):
    d = make([3300, 0, 3200], 1, 1, 128, 64, seed=24)
    assert is_cut(6500, 3, 1, 1, 128, 64)
    fresh = [1, 1, 1]
    ref = call(gpu, "chunked", d, fresh)
    d["state"].fill_(float("nan"))
    tokens = d["g"].shape[0]
    pad = torch.full((64, d["packed"].shape[1]), float("nan"), dtype=torch.bfloat16)
    d["packed"] = torch.cat([pad, d["packed"], pad])
    for x in ("g", "beta"):
        d[x] = torch.cat([torch.full((64, 1), float("nan")), d[x], torch.full((64, 1), float("nan"))])
    d["starts"] = [s + 64 for s in d["starts"]]
    out, state = call(gpu, "chunked", d, fresh)
    check({**d, "state": torch.nan_to_num(d["state"])}, out, torch.where(state.isnan(), 0.0, state), fresh)
    assert out[64:64 + tokens].isfinite().all() and ref[0].isfinite().all()
    assert sum(bool(s.isnan().all()) for s in state) == 2


def test_nan_stays_in_its_sequence_and_after_its_chunk(gpu):
    d = make([2000, 2500], 1, 1, 64, 32, seed=25)
    assert is_cut(4500, 2, 1, 1, 64, 32)
    clean = call(gpu, "chunked", d)
    d["packed"][700, 2 * 64] = float("nan")  # v of the first sequence's eleventh chunk
    out, state = call(gpu, "chunked", d)
    assert torch.equal(out[:640], clean[0][:640]) and torch.equal(out[2000:], clean[0][2000:])
    assert torch.equal(state[d["slots"][1]], clean[1][d["slots"][1]])
    assert torch.equal(out[:, :, 1:], clean[0][:, :, 1:])  # the other columns
    assert out[700:2000, :, 0].isnan().all()


def test_graph_reads_the_ranges_anew(gpu):
    hk, hv, dk, dv = 1, 1, 128, 64
    d = make([3000, 2600], hk, hv, dk, dv, seed=26)
    assert is_cut(5600, 2, hk, hv, dk, dv)
    q, k, v = heads(d, d["packed"].to(gpu))
    g, beta, first = d["g"].to(gpu), d["beta"].to(gpu), d["state"].to(gpu)
    starts = torch.tensor(d["starts"], dtype=torch.int32, device=gpu)
    slots, fresh = d["slots"].to(gpu), torch.zeros(2, dtype=torch.uint8, device=gpu)
    work = torch.zeros(bq.gated_delta_rule_workspace_bytes(5600, 2, hk, hv, dk, dv), dtype=torch.uint8, device=gpu)

    def run(out, state):
        bq.gated_delta_rule_chunked(q, k, v, g, beta, out, state, starts, work, slots=slots, fresh=fresh)

    out, state = torch.zeros(5600, hv, dv, dtype=torch.bfloat16, device=gpu), first.clone()
    run(out, state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, state)
    for i, middle in enumerate([3000, 64, 5600, 0, 2497]):
        fresh.fill_(i % 2)
        starts.copy_(torch.tensor([0, middle, 5600], dtype=torch.int32))
        want = torch.zeros_like(out), first.clone()
        run(*want)
        out.zero_()
        state.copy_(first)
        work.fill_(0xFF)  # NaN wherever it is read unwritten
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(state, want[1]), i
        d["starts"] = [0, middle, 5600]
        check(d, out.cpu(), state.cpu(), [i % 2] * 2)


def test_operands_beyond_the_caches(gpu):
    """So many chunks of heads that the lines of later ones are touched ahead: the same results at every end."""
    d = make([64 * 40 + 5, 64 * 31, 1, 64], 64, 64, 16, 64, seed=27)
    assert bq.gated_delta_rule_workspace_bytes(d["starts"][-1], 4, 64, 64, 16, 64) > 128 << 20
    check(d, *call(gpu, "chunked", d))


def test_longest_sequences_first(gpu):
    """More workgroups than start at once: equal lengths, empty sequences and slots outside keep their own results."""
    d = make([3, 130, 0, 130, 70, 1, 0], 8, 16, 128, 128, seed=28)
    d["slots"][4] = -1
    fresh = [0, 1, 1, 0, 1, 0, 0]
    check(d, *call(gpu, "chunked", d, fresh), fresh)
    want = call(gpu, "chunked", d, fresh)
    d["starts"] = [-9, *d["starts"][1:-1], 5000]
    got = call(gpu, "chunked", d, fresh)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("layout", ["odd rows", "odd start", "heads first"])
@pytest.mark.parametrize("tokens", [130, 2100])
def test_strides(gpu, layout, tokens):
    """The layouts of test_gpu_delta_rule's test at heads of 128, in one chain and in segments."""
    hk, hv, dk, dv = 1, 2, 128, 48
    d = make([tokens], hk, hv, dk, dv, seed=29, extra=1 if layout == "odd rows" else 16)
    plain = [x.contiguous().to(gpu) for x in heads(d, d["packed"])]
    if layout == "odd rows":
        other = list(heads(d, d["packed"].to(gpu)))
    elif layout == "odd start":
        other = []
        for x in plain:
            room = torch.zeros(x.numel() + 1, dtype=torch.bfloat16, device=gpu)
            room[1:].copy_(x.flatten())
            other.append(room[1:].view(x.shape))
    else:
        other = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in plain]
    results = []
    for qkv in (plain, other):
        out, state = torch.zeros(tokens, hv, dv, dtype=torch.bfloat16, device=gpu), d["state"].to(gpu)
        work = torch.zeros(bq.gated_delta_rule_workspace_bytes(tokens, 1, hk, hv, dk, dv), dtype=torch.uint8, device=gpu)
        bq.gated_delta_rule_chunked(*qkv, d["g"].to(gpu), d["beta"].to(gpu), out, state,
                                    torch.tensor([0, tokens], dtype=torch.int32, device=gpu), work,
                                    slots=d["slots"].to(gpu))
        results.append((out.cpu(), state.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    check(d, *results[0])
