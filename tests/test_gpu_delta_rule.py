"""The gated delta rule, recurrent and chunked, against the token-by-token definition in 64 bits.

Bounds, with u = 2^-24 and T the tokens a sequence took.  State: each token adds about eight independent roundings of
binary32 to it (two sums over dk, the decay, the update), so its relative error grows like 8 u sqrt(T + 4) in the
Frobenius norm.  Output: half a bf16 step, 2^-8 |o|, and 2^-13 of scale |q| times the largest column norm the state
has had (by Cauchy-Schwarz q^T S is off by no more than |q| times S's own error; the chunked form takes the output's
products from operands rounded to 2^-16)."""
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from delta_ref import delta_reference

pytestmark = pytest.mark.gpu
FORMS = ["recurrent", "chunked"]


def make(lens, hk, hv, dk, dv, seed, slots="permuted", l2norm=True, strong=False, extra=16):
    gen = torch.Generator().manual_seed(seed)
    tokens, count = sum(lens), len(lens)
    width = 2 * hk * dk + hv * dv + extra
    packed = torch.randn(tokens, width, generator=gen)
    if not l2norm and tokens:
        heads = packed[:, :2 * hk * dk].reshape(tokens, 2 * hk, dk)
        packed[:, :2 * hk * dk] = (heads / heads.norm(dim=-1, keepdim=True)).reshape(tokens, -1)
    packed = packed.bfloat16()
    g = -torch.exp(3 * torch.randn(tokens, hv, generator=gen) - 2)
    if strong:
        g = g * 30
    beta = torch.sigmoid(2 * torch.randn(tokens, hv, generator=gen))
    places = count + 2
    state = torch.randn(places, hv, dk, dv, generator=gen) * 0.1
    order = torch.randperm(places, generator=gen)[:count].to(torch.int32) if slots == "permuted" else None
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    return dict(packed=packed, g=g, beta=beta, state=state, slots=order, starts=starts, sizes=(hk, hv, dk, dv),
                l2norm=l2norm)


def heads(d, packed):
    hk, hv, dk, dv = d["sizes"]
    q = packed[:, :hk * dk].unflatten(1, (hk, dk))
    k = packed[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
    v = packed[:, 2 * hk * dk:2 * hk * dk + hv * dv].unflatten(1, (hv, dv))
    return q, k, v


def call(gpu, form, d, fresh=None, packed=None, scale=None, state=None):
    hk, hv, dk, dv = d["sizes"]
    q, k, v = heads(d, d["packed"].to(gpu) if packed is None else packed)
    tokens, count = d["starts"][-1], len(d["starts"]) - 1
    out = torch.full((d["g"].shape[0], hv, dv), 7.0, dtype=torch.bfloat16, device=gpu)
    state = d["state"].to(gpu) if state is None else state
    args = (q, k, v, d["g"].to(gpu), d["beta"].to(gpu), out, state,
            torch.tensor(d["starts"], dtype=torch.int32, device=gpu))
    kw = dict(slots=None if d["slots"] is None else d["slots"].to(gpu),
              fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.uint8, device=gpu), l2norm=d["l2norm"],
              scale=scale)
    if form == "recurrent":
        bq.gated_delta_rule_recurrent(*args, **kw)
    else:
        size = bq.gated_delta_rule_workspace_bytes(d["g"].shape[0], count, hk, hv, dk, dv)
        work = torch.full((size,), 0xFF, dtype=torch.uint8, device=gpu)  # NaN wherever it is read unwritten
        bq.gated_delta_rule_chunked(*args, work, **kw)
    torch.cuda.synchronize()
    return out.cpu(), state.cpu()


def check(d, out, state, fresh=None, scale=None):
    hk, hv, dk, dv = d["sizes"]
    scale = dk ** -0.5 if scale is None else scale
    q, k, v = heads(d, d["packed"])
    slots = None if d["slots"] is None else d["slots"].tolist()
    ref, ref_state, top = delta_reference(q, k, v, d["g"], d["beta"], d["state"], d["starts"], slots, fresh,
                                          d["l2norm"], scale)
    used = torch.zeros(out.shape[0], dtype=torch.bool)
    used[d["starts"][0]:d["starts"][-1]] = True
    assert (out[~used] == 7).all()
    qn = torch.ones(out.shape[0], hv, 1, dtype=torch.float64)
    if not d["l2norm"]:
        qn = q.double().norm(dim=-1).repeat_interleave(hv // hk, 1)[..., None]
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -13 * scale * qn * top
    off = (out.double() - ref).abs()
    assert (off[used] <= bound[used]).all(), (off[used] / bound[used].clamp_min(1e-300)).max()
    owned = {}
    for i in range(len(d["starts"]) - 1):
        owned[i if slots is None else slots[i]] = d["starts"][i + 1] - d["starts"][i]
    for s in range(state.shape[0]):
        if s not in owned:
            assert torch.equal(state[s].view(torch.int32), d["state"][s].view(torch.int32)), s
        else:
            n = ref_state[s].norm()
            err = (state[s].double() - ref_state[s]).norm()
            assert err <= 8 * 2.0 ** -24 * (owned[s] + 4) ** 0.5 * n, (s, float(err / n))


SIZES = [(1, 1, 128, 128), (2, 4, 128, 128), (1, 3, 64, 64), (2, 2, 64, 80), (1, 2, 48, 33), (1, 1, 1, 1), (1, 2, 8, 4),
         (2, 2, 100, 7), (1, 1, 65, 130), (3, 3, 127, 16)]
LENS = [[1], [2, 0, 3], [64], [63, 65, 1, 0], [130, 7], [257], [128, 192]]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", LENS, ids=lambda l: "-".join(map(str, l)))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_definition(gpu, form, sizes, lens):
    print(f"delta {form} {sizes} {lens}", flush=True)
    l2norm = (sum(lens) + sizes[3]) % 3 != 0
    d = make(lens, *sizes, seed=sum(lens) * 31 + sum(sizes), l2norm=l2norm)
    fresh = [i % 2 for i in range(len(lens))]
    check(d, *call(gpu, form, d, fresh), fresh)


@pytest.mark.parametrize("form", FORMS)
def test_long_sequence_without_decay(gpu, form):
    """g = 0 and beta near one: nothing is forgotten but by being written over; 700 tokens."""
    d = make([700], 1, 2, 128, 32, seed=5)
    d["g"].zero_()
    d["beta"] = 1 - d["beta"] * 0.05
    check(d, *call(gpu, form, d))


@pytest.mark.parametrize("form", FORMS)
def test_keys_that_repeat(gpu, form):
    """The same key again and again with beta = 1: the triangular system at its worst."""
    d = make([200], 1, 1, 64, 32, seed=6)
    d["packed"][:, 64:128] = d["packed"][:1, 64:128]
    d["beta"].fill_(1.0)
    d["g"].mul_(0.01)
    check(d, *call(gpu, form, d))


@pytest.mark.parametrize("form", FORMS)
def test_strong_decay_and_forgetting(gpu, form):
    """Decays far below exp's range next to weak ones, and g = -infinity: the state is gone, nothing is NaN."""
    d = make([150, 70], 1, 4, 128, 48, seed=7, strong=True)
    d["g"][40, 0] = d["g"][41, 0] = d["g"][149, 1] = d["g"][150, 2] = float("-inf")
    out, state = call(gpu, form, d)
    assert out.isfinite().all() and state.isfinite().all()
    check(d, out, state)


@pytest.mark.parametrize("form", FORMS)
def test_beta_zero_and_one_and_zero_vectors(gpu, form):
    d = make([90, 5], 1, 2, 64, 16, seed=8)
    d["beta"][::3] = 0
    d["beta"][1::3] = 1
    d["packed"][10:14] = 0
    check(d, *call(gpu, form, d))


@pytest.mark.parametrize("form", FORMS)
def test_slots_absent_and_outside(gpu, form):
    """slots = None is the sequence's own number; a slot outside the state starts from zeros and is not kept."""
    d = make([66, 3, 1], 1, 2, 64, 32, seed=9, slots=None)
    check(d, *call(gpu, form, d))
    d["slots"] = torch.tensor([-1, 4, 5], dtype=torch.int32)  # five slots: 0..4
    check(d, *call(gpu, form, d))


@pytest.mark.parametrize("form", FORMS)
def test_nothing_reads_a_fresh_slot_or_a_foreign_token(gpu, form):
    """NaN in the slots of fresh sequences, in slots of nobody and in tokens of no sequence reaches nothing."""
    d = make([70, 0, 65], 1, 2, 128, 64, seed=10)
    fresh = [1, 1, 1]
    ref = call(gpu, form, d, fresh)
    d["state"].fill_(float("nan"))
    tokens = d["g"].shape[0]
    pad = torch.full((9, d["packed"].shape[1]), float("nan"), dtype=torch.bfloat16)
    d["packed"] = torch.cat([pad, d["packed"], pad])
    for x in ("g", "beta"):
        d[x] = torch.cat([torch.full((9, 2), float("nan")), d[x], torch.full((9, 2), float("nan"))])
    d["starts"] = [s + 9 for s in d["starts"]]
    out, state = call(gpu, form, d, fresh)
    assert torch.equal(out[9:9 + tokens], ref[0]) and (out[:9] == 7).all() and (out[9 + tokens:] == 7).all()
    for s in d["slots"].tolist():
        assert torch.equal(state[s], ref[1][s])
    assert sum(bool(s.isnan().all()) for s in state) == 2


@pytest.mark.parametrize("form", FORMS)
def test_nan_stays_in_its_sequence_and_head(gpu, form):
    d = make([67, 70, 3], 1, 2, 64, 32, seed=11)
    clean = call(gpu, form, d)
    d["packed"][80, 2 * 64] = float("nan")  # v of head 0, second sequence
    out, state = call(gpu, form, d)
    same = [0, 2]
    assert torch.equal(out[:67], clean[0][:67]) and torch.equal(out[137:], clean[0][137:])
    assert torch.equal(out[:, 1], clean[0][:, 1])
    for i in same:
        assert torch.equal(state[d["slots"][i]], clean[1][d["slots"][i]])
    assert state[d["slots"][1], 0].isnan().any()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layout", ["odd rows", "odd start", "heads first", "shared head"])
def test_strides(gpu, form, layout):
    """Rows of odd length, a first value at an odd place, [heads, tokens, d] storage, and a head expanded over
    several (stride zero) give what contiguous tensors give."""
    hk, hv, dk, dv = 2, 4, 64, 48
    d = make([65, 20], hk, hv, dk, dv, seed=12, extra=1 if layout == "odd rows" else 16)
    q, k, v = (x.contiguous() for x in heads(d, d["packed"]))
    if layout == "shared head":
        q = q[:, :1].expand(-1, hk, -1)
    plain = [x.contiguous().to(gpu) for x in (q, k, v)]
    if layout == "odd rows":
        other = list(heads(d, d["packed"].to(gpu)))
    elif layout == "odd start":
        other = []
        for x in plain:
            room = torch.zeros(x.numel() + 1, dtype=torch.bfloat16, device=gpu)
            room[1:].copy_(x.flatten())
            other.append(room[1:].view(x.shape))
    elif layout == "heads first":
        other = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in plain]
    else:
        other = [plain[0][:, :1].expand(-1, hk, -1), *plain[1:]]
    results = []
    for qkv in (plain, other):
        out = torch.zeros(85, hv, dv, dtype=torch.bfloat16, device=gpu)
        state = d["state"].to(gpu)
        args = (*qkv, d["g"].to(gpu), d["beta"].to(gpu), out, state, torch.tensor([0, 65, 85], dtype=torch.int32, device=gpu))
        if form == "recurrent":
            bq.gated_delta_rule_recurrent(*args)
        else:
            work = torch.zeros(bq.gated_delta_rule_workspace_bytes(85, 2, hk, hv, dk, dv), dtype=torch.uint8, device=gpu)
            bq.gated_delta_rule_chunked(*args, work)
        results.append((out.cpu(), state.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("form", FORMS)
def test_scale_and_no_tokens(gpu, form):
    d = make([70], 1, 1, 64, 16, seed=13)
    check(d, *call(gpu, form, d, scale=0.5), scale=0.5)
    # no tokens at all: a fresh sequence's state becomes zero, the other stays
    d = make([0, 0], 1, 1, 64, 16, seed=14)
    out, state = call(gpu, form, d, [1, 0])
    assert not state[d["slots"][0]].any() and torch.equal(state[d["slots"][1]], d["state"][d["slots"][1]])


@pytest.mark.parametrize("form", FORMS)
def test_ranges_beyond_the_tokens_are_cut_off(gpu, form):
    """starts is device data: what lies outside the tokens is cut off, a range that runs backwards is empty."""
    d = make([70, 30], 1, 2, 64, 16, seed=15)
    want = call(gpu, form, d)
    d["starts"] = [-5, 70, 1000]
    got = call(gpu, form, d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("form", FORMS)
def test_many_sequences(gpu, form):
    """Enough sequences that a chunk's own is found past the first few hundred."""
    lens = [(i * 7) % 5 for i in range(600)]
    lens[333] = 129
    d = make(lens, 1, 1, 16, 8, seed=16)
    fresh = [int(i % 3 == 0) for i in range(600)]
    check(d, *call(gpu, form, d, fresh), fresh)


def test_forms_agree_when_a_prompt_is_continued(gpu):
    """A prompt in two chunked calls and then single tokens, against one chunked call: the state carries over."""
    d = make([200], 2, 4, 128, 64, seed=17)
    whole = call(gpu, "chunked", d)
    q, k, v = heads(d, d["packed"].to(gpu))
    state, out = d["state"].to(gpu), torch.zeros(200, 4, 64, dtype=torch.bfloat16, device=gpu)
    g, beta, slots = d["g"].to(gpu), d["beta"].to(gpu), d["slots"].to(gpu)
    for a, b in [(0, 100), (100, 190), *((t, t + 1) for t in range(190, 200))]:
        starts = torch.tensor([0, b - a], dtype=torch.int32, device=gpu)
        args = (q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], out[a:b], state, starts)
        if b - a > 1:
            work = torch.zeros(bq.gated_delta_rule_workspace_bytes(b - a, 1, 2, 4, 128, 64), dtype=torch.uint8, device=gpu)
            bq.gated_delta_rule_chunked(*args, work, slots=slots)
        else:
            bq.gated_delta_rule_recurrent(*args, slots=slots)
    torch.cuda.synchronize()
    check(d, out.cpu(), state.cpu())
    check(d, *whole)


@pytest.mark.parametrize("form", FORMS)
def test_stream_and_graph(gpu, form):
    """On a side stream and captured in a graph: the same bits; the graph reads starts, slots and fresh anew at each
    replay."""
    hk, hv, dk, dv = 1, 2, 128, 64
    d = make([90, 40], hk, hv, dk, dv, seed=18)
    q, k, v = heads(d, d["packed"].to(gpu))
    g, beta = d["g"].to(gpu), d["beta"].to(gpu)
    starts = torch.tensor(d["starts"], dtype=torch.int32, device=gpu)
    slots, fresh = d["slots"].to(gpu), torch.zeros(2, dtype=torch.uint8, device=gpu)
    first = d["state"].to(gpu)
    work = torch.zeros(bq.gated_delta_rule_workspace_bytes(130, 2, hk, hv, dk, dv), dtype=torch.uint8, device=gpu)

    def run(out, state):
        args = (q, k, v, g, beta, out, state, starts)
        if form == "recurrent":
            bq.gated_delta_rule_recurrent(*args, slots=slots, fresh=fresh)
        else:
            bq.gated_delta_rule_chunked(*args, work, slots=slots, fresh=fresh)

    def eager():
        out, state = torch.zeros(130, hv, dv, dtype=torch.bfloat16, device=gpu), first.clone()
        run(out, state)
        return out, state

    want = eager()
    out, state = torch.zeros_like(want[0]), first.clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run(out, state)
    stream.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(state, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, state)
    for i in range(4):
        fresh.fill_(i % 2)
        starts.copy_(torch.tensor([0, 90 - i, 130], dtype=torch.int32))
        slots.copy_(slots.flip(0))
        want = eager()
        out.zero_()
        state.copy_(first)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(state, want[1]), i
