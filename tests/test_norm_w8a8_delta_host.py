"""Host-side refusals (no GPU) of the norms, the int8 product and the gated delta rule: the C ABI's argument checks,
which run before any HIP call, and the binding's checks of types, shapes and sizes."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def bq():
    import os
    import bit_quantized_matmul_quantize_amd as m
    if not os.path.exists(m.LIB_PATH):
        from bit_quantized_matmul_quantize_amd import build
        build.build()
    return m


P = ctypes.c_void_p


def at(i):
    return P(0x10000000 * i)  # fake device addresses, far apart: every call below is refused before they are used


A, B, C, D, MIS, ODD = at(1), at(2), at(3), at(4), P(0x10000008), P(0x10000001)

NORMS = ("add_rms_norm_bf16", "add_rms_norm_quantize_q8_1", "add_rms_norm_quantize_int8")


@pytest.mark.parametrize("name", NORMS)
@pytest.mark.parametrize("args,status,needle", [
    ((None, B, C, D, 4, 64, 1e-6, None), -1, "null"),
    ((A, B, None, D, 4, 64, 1e-6, None), -1, "null"),
    ((A, B, C, None, 4, 64, 1e-6, None), -1, "null"),
    ((A, B, C, D, 0, 64, 1e-6, None), -1, "m=0"),
    ((A, B, C, D, 4, 0, 1e-6, None), -1, "k=0"),
    ((A, B, C, D, 4, (1 << 30) + 1, 1e-6, None), -1, "too large"),
    ((A, B, C, D, 1 << 31, 64, 1e-6, None), -1, "too large"),
    ((A, B, C, D, 4, 64, -1.0, None), -1, "eps"),
    ((A, B, C, D, 4, 64, float("nan"), None), -1, "eps"),
    ((MIS, B, C, D, 4, 64, 1e-6, None), -3, "aligned"),
    ((A, MIS, C, D, 4, 64, 1e-6, None), -3, "aligned"),
    ((A, B, C, A, 4, 64, 1e-6, None), -1, "overlaps the input"),
    ((A, B, C, B, 4, 64, 1e-6, None), -1, "overlaps the residual"),
    ((A, B, C, C, 4, 64, 1e-6, None), -1, "overlaps the weight"),
    ((A, A, C, D, 4, 64, 1e-6, None), -1, "residual overlaps"),
])
def test_norm_refusals(bq, name, args, status, needle):
    assert getattr(bq.lib(), name)(*args) == status
    assert needle in bq.lib().bq_last_error().decode()


@pytest.mark.parametrize("call,status,needle", [
    (lambda l: l.quantize_rows_int8(None, B, 4, 64, None), -1, "null"),
    (lambda l: l.quantize_rows_int8(A, B, 0, 64, None), -1, "rows=0"),
    (lambda l: l.quantize_rows_int8(A, B, 4, (1 << 30) + 1, None), -1, "too large"),
    (lambda l: l.quantize_rows_int8(A, MIS, 4, 64, None), -3, "aligned"),
    (lambda l: l.quantize_rows_int8(A, P(0x10000000 + 256), 4, 64, None), -1, "overlaps"),
    (lambda l: l.w8a8_gemm(A, B, None, None, 4, 64, 64, None), -1, "null"),
    (lambda l: l.w8a8_gemm(A, B, None, C, 0, 64, 64, None), -1, "m=0"),
    (lambda l: l.w8a8_gemm(A, B, None, C, 4, 0, 64, None), -1, "n=0"),
    (lambda l: l.w8a8_gemm(A, B, None, C, 4, 64, 0, None), -1, "k=0"),
    (lambda l: l.w8a8_gemm(A, B, None, C, 4, 64, 131072, None), -1, "131071"),
    (lambda l: l.w8a8_gemm(A, B, None, C, 4, 65535 * 128 + 1, 64, None), -1, "too large"),
    (lambda l: l.w8a8_gemm(A, B, None, MIS, 4, 64, 64, None), -3, "aligned"),
    (lambda l: l.w8a8_gemm(A, B, ODD, C, 4, 64, 64, None), -3, "bias"),
    (lambda l: l.w8a8_gemm(A, B, None, A, 4, 64, 64, None), -1, "overlaps the activations"),
    (lambda l: l.w8a8_gemm(A, B, None, B, 4, 64, 64, None), -1, "overlaps the weight"),
    (lambda l: l.w8a8_gemm(A, B, P(0x30000000 + 16), C, 4, 64, 64, None), -1, "overlaps the bias"),
])
def test_int8_refusals(bq, call, status, needle):
    assert call(bq.lib()) == status
    assert needle in bq.lib().bq_last_error().decode()


def delta_args(**change):
    d = dict(q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), out=at(6), state=at(7), starts=at(8), slots=at(9),
             fresh=at(10), tokens=70, count=2, state_slots=3, hk=2, hv=4, dk=64, dv=32, q_token=128, q_head=64,
             k_token=128, k_head=64, v_token=128, v_head=32, scale=0.125, l2norm=1, stream=None)
    d.update(change)
    return d


DELTA = [
    (dict(q=None), -1, "null"), (dict(beta=None), -1, "null"), (dict(out=None), -1, "null"),
    (dict(starts=None), -1, "null"), (dict(state=None), -1, "null state"),
    (dict(hk=0), -1, "hk=0"), (dict(hk=3), -1, "must divide"), (dict(dk=0), -1, "dk=0"), (dict(dv=0), -1, "dv=0"),
    (dict(dk=129), -2, "129"), (dict(hv=65536, hk=1), -1, "too large"), (dict(tokens=1 << 31), -1, "too large"),
    (dict(count=(1 << 31) - 1), -1, "too large"),
    (dict(q=ODD), -3, "2-byte"), (dict(g=P(0x40000002)), -3, "4-byte"), (dict(state=P(0x70000002)), -3, "4-byte"),
    (dict(q_token=1 << 62), -1, "strides of q"), (dict(v_head=(1 << 64) - 1), -1, "strides of v"),
    (dict(out=at(1)), -1, "overlaps q"), (dict(out=at(4)), -1, "overlaps g"), (dict(state=at(3)), -1, "overlaps v"),
    (dict(state=at(6)), -1, "overlaps the output"), (dict(state=at(8)), -1, "overlaps starts"),
    (dict(state=at(9)), -1, "overlaps slots"), (dict(out=at(8)), -1, "overlaps starts"),
    (dict(out=at(10)), -1, "overlaps fresh"),
    # q's rows lie apart: it is the strides that make it reach the output
    (dict(q_token=0x50000000 // 2 // 69), -1, "overlaps q"),
]


@pytest.mark.parametrize("change,status,needle", DELTA)
@pytest.mark.parametrize("chunked", [False, True])
def test_delta_refusals(bq, chunked, change, status, needle):
    d = delta_args(**change)
    v = list(d.values())
    if chunked:
        v[10:10] = [at(12), 1 << 28]
        got = bq.lib().gated_delta_rule_chunked(*v)
    else:
        got = bq.lib().gated_delta_rule_recurrent(*v)
    assert got == status
    assert needle in bq.lib().bq_last_error().decode()


@pytest.mark.parametrize("workspace,size,status,needle", [
    (None, 1 << 28, -1, "null workspace"), (at(12), 100, -1, "are needed"), (P(0x1008), 1 << 28, -3, "16-byte"),
    (at(7), 1 << 28, -1, "overlaps the state"), (at(2), 1 << 28, -1, "overlaps k"),
    (at(9), 1 << 28, -1, "overlaps slots"),
])
def test_chunked_workspace_refusals(bq, workspace, size, status, needle):
    v = list(delta_args().values())
    v[10:10] = [workspace, size]
    assert bq.lib().gated_delta_rule_chunked(*v) == status
    assert needle in bq.lib().bq_last_error().decode()


def test_empty_batch_is_no_error(bq):
    v = list(delta_args(count=0, tokens=0, q=None, k=None, v=None, g=None, beta=None, out=None).values())
    assert bq.lib().gated_delta_rule_recurrent(*v) == 0


def test_sizes(bq):
    assert bq.int8_rows_bytes(3, 1) == 3 * 132 and bq.int8_rows_bytes(5, 129) == 5 * 260
    assert bq.int8_rows_bytes(4096, 17408) == 4096 * 17412 and bq.int8_rows_bytes(1, (1 << 30) + 1) == 0
    assert bq.gated_delta_rule_workspace_bytes(64, 1, 2, 3, 64, 64) == 0  # hk does not divide hv
    assert bq.gated_delta_rule_workspace_bytes(64, 1, 1, 1, 129, 64) == 0
    big, small = (bq.gated_delta_rule_workspace_bytes(t, 1, 16, 32, 128, 128) for t in (16384, 64))
    assert 0 < small < big


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


def test_binding_checks_sizes_and_types(bq):
    m, k, n = 3, 130, 17
    rows = bq.int8_rows_bytes
    short = [
        (lambda: bq.add_rms_norm_bf16(bf(m * k - 1), None, bf(k), bf(m * k), m, k), "x"),
        (lambda: bq.add_rms_norm_bf16(bf(m * k), bf(m * k - 1), bf(k), bf(m * k), m, k), "residual"),
        (lambda: bq.add_rms_norm_bf16(bf(m * k), None, bf(k - 1), bf(m * k), m, k), "weight"),
        (lambda: bq.add_rms_norm_bf16(bf(m * k), None, bf(k), bf(m * k - 1), m, k), "out"),
        (lambda: bq.add_rms_norm_quantize_q8_1(bf(m * k), None, bf(k), u8(bq.q8_1_act_bytes(m, k) - 1), m, k), "out_q8"),
        (lambda: bq.add_rms_norm_quantize_int8(bf(m * k), None, bf(k), u8(rows(m, k) - 1), m, k), "out_i8"),
        (lambda: bq.quantize_rows_int8(bf(m * k), u8(rows(m, k) - 1), m, k), "out_i8"),
        (lambda: bq.w8a8_gemm(u8(rows(m, k) - 1), u8(rows(n, k)), bf(m * n), m, n, k), "act_i8"),
        (lambda: bq.w8a8_gemm(u8(rows(m, k)), u8(rows(n, k) - 1), bf(m * n), m, n, k), "w_i8"),
        (lambda: bq.w8a8_gemm(u8(rows(m, k)), u8(rows(n, k)), bf(m * n), m, n, k, bias=bf(n - 1)), "bias"),
    ]
    for call, what in short:
        with pytest.raises(ValueError) as e:
            call()
        assert str(e.value).startswith(what + ":") and "address" in str(e.value)
    with pytest.raises(TypeError, match="bfloat16"):
        bq.add_rms_norm_bf16(torch.zeros(m * k), None, bf(k), bf(m * k), m, k)
    with pytest.raises(ValueError, match="device tensor"):
        bq.w8a8_gemm(u8(rows(m, k)), u8(rows(n, k)), bf(m * n), m, n, k)


def test_binding_checks_delta_shapes(bq):
    t, hk, hv, dk, dv, c = 5, 1, 2, 16, 24, 2
    ok = dict(q=bf(t, hk, dk), k=bf(t, hk, dk), v=bf(t, hv, dv), g=torch.zeros(t, hv), beta=torch.zeros(t, hv),
              out=bf(t, hv, dv), state=torch.zeros(c, hv, dk, dv), starts=torch.zeros(c + 1, dtype=torch.int32))
    for change, err, needle in [
        (dict(q=bf(t, dk)), ValueError, "tokens, heads"),
        (dict(k=bf(t, hk, dk + 1)), ValueError, "k:"),
        (dict(v=bf(t + 1, hv, dv)), ValueError, "v:"),
        (dict(g=torch.zeros(t, hv, dtype=torch.float64)), TypeError, "g:"),
        (dict(beta=torch.zeros(t, hv + 1)), ValueError, "beta:"),
        (dict(out=torch.zeros(t, hv, dv)), TypeError, "out:"),
        (dict(state=torch.zeros(c, hv, dv, dk)), ValueError, "state:"),
        (dict(state=torch.zeros(c - 1, hv, dk, dv)), ValueError, "device tensor|slots for"),
        (dict(starts=torch.zeros(c + 1, dtype=torch.int64)), TypeError, "starts:"),
        (dict(slots=torch.zeros(c + 1, dtype=torch.int32)), ValueError, "slots:"),
        (dict(fresh=torch.zeros(c, dtype=torch.bool)), TypeError, "fresh:"),
        (dict(), ValueError, "device tensor"),
    ]:
        with pytest.raises(err, match=needle):
            bq.gated_delta_rule_recurrent(**{**ok, **change})
    with pytest.raises(TypeError, match="workspace"):
        bq.gated_delta_rule_chunked(**ok, workspace=bf(16))


def chunked_need(bq, tokens, count, hk, hv, dk, dv):
    """What the call itself asks for, from its refusal of a workspace of one byte."""
    v = list(delta_args(tokens=tokens, count=count, hk=hk, hv=hv, dk=dk, dv=dv, q=at(1 << 10), k=at(1 << 11), v=at(1 << 12),
                        g=at(1 << 13), beta=at(1 << 14), out=at(1 << 15), state=at(1 << 16), starts=at(1 << 17), slots=None,
                        fresh=None, state_slots=count, q_token=hk * dk, q_head=dk, k_token=hk * dk, k_head=dk,
                        v_token=hv * dv, v_head=dv).values())
    v[10:10] = [at(12), 1]
    assert bq.lib().gated_delta_rule_chunked(*v) == -1
    return int(bq.lib().bq_last_error().decode().split(", ")[1].split()[0])


def test_a_workspace_for_the_largest_call_serves_every_smaller_one(bq):
    """A program allocates once, for its most tokens and its most sequences."""
    import random
    rng = random.Random(5)
    size = bq.gated_delta_rule_workspace_bytes
    fixed = [(8192, 4, 8192, 1, (4, 4, 128, 128)), (7104, 1, 7040, 1, (16, 16, 128, 128)), (16384, 8, 7000, 1, (1, 1, 64, 64))]
    for i in range(600):
        hk = rng.choice([1, 1, 2, 4, 8, 16])
        heads = (hk, hk * rng.choice([1, 2]), rng.choice([1, 33, 64, 65, 128]), rng.choice([1, 7, 64, 80, 128, 130]))
        tokens, count = int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 5))
        less, fewer = rng.randint(1, tokens), rng.randint(1, count)
        if i < len(fixed):
            tokens, count, less, fewer, heads = fixed[i]
        assert size(less, fewer, *heads) <= size(tokens, count, *heads), (tokens, count, less, fewer, heads)
        need = chunked_need(bq, less, fewer, *heads)
        assert 0 < need <= size(less, fewer, *heads)


@pytest.mark.parametrize("tokens,count,heads,cut", [
    (8192, 1, 1, True), (9000, 1, 4, True), (16000, 1, 8, True), (16000, 2, 2, True),
    # measured slower in every cut: 476 us at best and 413 in one chain, 192 (in 32s) and 176, 756 and 622
    (16000, 1, 16, False), (6500, 1, 16, False), (24000, 1, 16, False), (2500, 1, 16, False), (16384, 1, 32, False),
])
def test_long_sequences_are_cut_where_that_measured_faster(bq, tokens, count, heads, cut):
    sizes = (heads, heads, 128, 128)
    chunk = chunked_need(bq, 1, 1, *sizes)  # one chunk of all heads
    assert (chunked_need(bq, tokens, count, *sizes) > (tokens // 64 + count) * chunk) == cut


@pytest.mark.parametrize("k,rows", [(512, 1 << 26), (64, (1 << 31) - 1), (513, 1 << 25), (4096, 1 << 23), (70000, 1 << 23)])
def test_more_threads_than_a_launch_has_are_refused(bq, k, rows):
    """A launch's threads are counted in 32 bits."""
    far = [at(1 << i) for i in (20, 21, 22, 23)]
    for name in NORMS:
        assert getattr(bq.lib(), name)(far[0], far[1], far[2], far[3], rows, k, 1e-6, None) == -1
        assert "too large" in bq.lib().bq_last_error().decode()
    assert bq.lib().quantize_rows_int8(far[0], far[3], rows, k, None) == -1
    assert "too large" in bq.lib().bq_last_error().decode()


@pytest.mark.parametrize("chunked,change", [
    (False, dict(count=1 << 24, hk=1, hv=4, dv=32)), (False, dict(count=1 << 19, hk=1, hv=32, dv=128)),
    (True, dict(count=1 << 15, hk=1, hv=32, dv=128)), (True, dict(count=1 << 21, hk=1, hv=4, dv=16)),
    (True, dict(tokens=1 << 30, count=1, hk=1, hv=1, dv=1)), (True, dict(tokens=64, count=(1 << 24) - 16, hk=1, hv=1, dv=1, dk=1)),
])
def test_more_threads_than_a_delta_launch_has_are_refused(bq, chunked, change):
    far = {k: at(1 << (20 + i)) for i, k in enumerate(("q", "k", "v", "g", "beta", "out", "state", "starts"))}
    v = list(delta_args(**far, slots=None, fresh=None, state_slots=1, **change).values())
    if chunked:
        v[10:10] = [at(12), 1 << 62]
    fn = bq.lib().gated_delta_rule_chunked if chunked else bq.lib().gated_delta_rule_recurrent
    assert fn(*v) == -1
    assert "too large" in bq.lib().bq_last_error().decode()


def test_int8_rows_bytes_is_the_librarys(bq):
    for rows in (1, 2, 3, 4096, (1 << 31) - 1):
        for k in (1, 127, 128, 129, 2563, 131071, 1 << 30, (1 << 30) + 1, (1 << 32) - 1):
            assert bq.int8_rows_bytes(rows, k) == bq.lib().int8_rows_bytes(rows, k), (rows, k)
