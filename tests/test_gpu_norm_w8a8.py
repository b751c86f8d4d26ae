"""The norms with bf16, q8_1 and int8 outputs, the int8 row quantizer and the int8 product against 64-bit
definitions.

Bounds.  Codes, residuals and the q8_1 bytes are exact.  Scales: one rounding to binary32, 2^-24, and the reference's
own: 2^-23.  bf16 results: half a bf16 step, 2^-8 |y|, and for the product four roundings in binary32 before it (the
sum's conversion, two scales, the bias): 2^-22 of |sum sa sw| + |bias|."""
import numpy as np
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq

pytestmark = pytest.mark.gpu
EPS = 1e-6


def rows_of(buf, rows, k):
    kp = (k + 127) // 128 * 128
    return buf[:rows * kp].view(torch.int8).view(rows, kp), buf[rows * kp:rows * (kp + 4)].view(torch.float32)


def make(m, k, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(spread * torch.randn(m, 1, generator=g))
    r = 3 * torch.randn(m, k, generator=g)
    w = 1 + 0.2 * torch.randn(k, generator=g)
    return x.bfloat16(), r.bfloat16(), w.bfloat16()


def norm_reference(x, r, w):
    h = x if r is None else (x.float() + r.float()).bfloat16()
    hd = h.double()
    root = torch.sqrt((hd * hd).mean(1, keepdim=True) + EPS)
    t = hd * w.double()
    return h, t, root


def codes_reference(t):
    top = t.abs().amax(1, keepdim=True)
    return torch.where(top > 0, torch.round(127 * t / torch.where(top > 0, top, 1.0)), 0.0).to(torch.int8), top


SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 127), (2, 129), (33, 255), (4, 257), (7, 2563), (3, 4096), (2, 4104),
          (2, 5120), (2, 8200), (2, 17408), (1, 32768), (2, 32771), (1, 70001)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k", SHAPES)
def test_norm_outputs(gpu, m, k, residual):
    print(f"norm m={m} k={k} residual={residual}", flush=True)
    x, r, w = make(m, k, 100 + m + k)
    if m > 2:
        x[1] = 0
        r[1] = 0
    xd, wd = x.to(gpu), w.to(gpu)
    h, t, root = norm_reference(x, r if residual else None, w)
    codes, top = codes_reference(t)

    rd = r.to(gpu) if residual else None
    out = torch.full((m, k), 7.0, dtype=torch.bfloat16, device=gpu)
    bq.add_rms_norm_bf16(xd, rd, wd, out, m, k, EPS)
    y = t / root
    assert ((out.cpu().double() - y).abs() <= (2.0 ** -8 + 2.0 ** -23) * y.abs()).all()
    if residual:
        assert torch.equal(rd.cpu(), h)

    rd = r.to(gpu) if residual else None
    q8 = torch.full((bq.q8_1_act_bytes(m, k),), 0xAA, dtype=torch.uint8, device=gpu)
    q8_two = torch.full_like(q8, 0x55)
    bq.add_rms_norm_quantize_q8_1(xd, rd, wd, q8, m, k, EPS)
    bq.quantize_act_q8_1(out, q8_two, m, k)
    assert torch.equal(q8, q8_two)
    if residual:
        assert torch.equal(rd.cpu(), h)

    rd = r.to(gpu) if residual else None
    i8 = torch.full((bq.int8_rows_bytes(m, k),), 0xAA, dtype=torch.uint8, device=gpu)
    bq.add_rms_norm_quantize_int8(xd, rd, wd, i8, m, k, EPS)
    c, s = rows_of(i8.cpu(), m, k)
    assert torch.equal(c[:, :k], codes) and not c[:, k:].any()
    ref = (top / root / 127)[:, 0]
    assert ((s.double() - ref).abs() <= 2.0 ** -23 * ref).all()
    if residual:
        assert torch.equal(rd.cpu(), h)


@pytest.mark.parametrize("rows,k", [(1, 1), (3, 130), (17, 2048), (2, 17408), (1, 40000)])
def test_row_quantizer(gpu, rows, k):
    x, _, _ = make(rows, k, 300 + k)
    buf = torch.full((bq.int8_rows_bytes(rows, k),), 0xAA, dtype=torch.uint8, device=gpu)
    bq.quantize_rows_int8(x.to(gpu), buf, rows, k)
    codes, top = codes_reference(x.double())
    c, s = rows_of(buf.cpu(), rows, k)
    assert torch.equal(c[:, :k], codes) and not c[:, k:].any()
    assert ((s.double() - top[:, 0] / 127).abs() <= 2.0 ** -23 * top[:, 0] / 127).all()


def test_every_tie_goes_to_even(gpu):
    # top = 254: 127 x / top = x / 2, a tie for every odd x
    x = torch.cat([torch.tensor([254.0]), torch.arange(-254.0, 255.0)]).bfloat16()[None]
    k = x.shape[1]
    buf = torch.zeros(bq.int8_rows_bytes(1, k), dtype=torch.uint8, device=gpu)
    bq.quantize_rows_int8(x.to(gpu), buf, 1, k)
    want = np.rint(x.double().numpy() / 2).astype(np.int8)
    assert np.array_equal(rows_of(buf.cpu(), 1, k)[0][:, :k].numpy(), want)


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -60, 2.0 ** 60, 2.0 ** 126])
def test_far_scales(gpu, scale):
    """Rows near the ends of binary32: no product on the way overflows, codes stay exact."""
    x = (make(4, 300, 9, 0.0)[0].double() * scale).bfloat16()
    x = torch.where(x.isinf(), torch.sign(x) * 3e38, x.float()).bfloat16()
    buf = torch.zeros(bq.int8_rows_bytes(4, 300), dtype=torch.uint8, device=gpu)
    bq.quantize_rows_int8(x.to(gpu), buf, 4, 300)
    codes, top = codes_reference(x.double())
    c, s = rows_of(buf.cpu(), 4, 300)
    assert torch.equal(c[:, :300], codes)
    # a scale below the normal range of binary32 is off by half a step of 2^-149
    assert ((s.double() - top[:, 0] / 127).abs() <= 2.0 ** -23 * top[:, 0] / 127 + 2.0 ** -150).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_with_nan_or_infinity_keep_to_themselves(gpu, bad):
    m, k = 3, 1000
    x, r, w = make(m, k, 77)
    x[1, 500] = bad
    clean = x.clone()
    clean[1] = 1
    outs = []
    for a in (x, clean):
        i8 = torch.zeros(bq.int8_rows_bytes(m, k), dtype=torch.uint8, device=gpu)
        bf = torch.zeros(m, k, dtype=torch.bfloat16, device=gpu)
        bq.add_rms_norm_quantize_int8(a.to(gpu), r.to(gpu), w.to(gpu), i8, m, k, EPS)
        bq.add_rms_norm_bf16(a.to(gpu), r.to(gpu), w.to(gpu), bf, m, k, EPS)
        outs.append((*rows_of(i8.cpu(), m, k), bf.cpu()))
    (c, s, y), (c2, s2, y2) = outs
    keep = [0, 2]
    assert torch.equal(c[keep], c2[keep]) and torch.equal(s[keep], s2[keep]) and torch.equal(y[keep], y2[keep])
    assert s[1].isnan() and not c[1].any() and y[1, 500].isnan()


def product_case(m, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    bufs = []
    for rows in (m, n):
        kp = (k + 127) // 128 * 128
        codes = torch.randint(-127, 128, (rows, k), generator=g, dtype=torch.int8)
        scale = torch.exp(2 * torch.randn(rows, generator=g)) * 0.01
        buf = torch.zeros(rows * (kp + 4), dtype=torch.uint8)
        buf[:rows * kp].view(torch.int8).view(rows, kp)[:, :k] = codes
        buf[rows * kp:].view(torch.float32).copy_(scale)
        bufs.append((buf, codes, scale))
    bias = torch.randn(n, generator=g).bfloat16()
    return bufs, bias


def check_product(out, bufs, bias):
    (_, a, sa), (_, w, sw) = bufs
    # sums of code products are whole numbers below 2^31: exact in binary64
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    y = p if bias is None else p + bias.double()
    extra = 0 if bias is None else bias.double().abs()
    assert ((out.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2.0 ** -22 * (p.abs() + extra)).all()


PRODUCTS = [(1, 1, 1), (1, 64, 64), (1, 1000, 2048), (2, 33, 130), (3, 16, 128), (5, 257, 384), (8, 513, 1000),
            (9, 100, 4096), (15, 2048, 129), (16, 640, 512), (17, 300, 2563), (31, 129, 640), (33, 96, 896),
            (63, 512, 2048), (64, 1111, 777), (65, 64, 64), (127, 200, 256), (128, 384, 1024), (129, 1, 5120),
            (200, 515, 300), (256, 256, 128), (257, 1025, 130), (300, 4133, 2563), (511, 768, 5120), (1025, 300, 512),
            (2049, 511, 384), (1, 5120, 17408), (8, 700, 17408), (1, 3, 131071)]


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(gpu, m, n, k, with_bias):
    print(f"w8a8 m={m} n={n} k={k} bias={with_bias}", flush=True)
    bufs, bias = product_case(m, n, k, m * 7 + n * 3 + k)
    bias = bias if with_bias else None
    # guard values around the output
    out = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device=gpu)
    view = out[32:32 + m * n].view(m, n)
    bq.w8a8_gemm(bufs[0][0].to(gpu), bufs[1][0].to(gpu), view, m, n, k, bias=None if bias is None else bias.to(gpu))
    assert (out[:32] == 7).all() and (out[32 + m * n:] == 7).all()
    check_product(view.cpu(), bufs, bias)


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (16, 300, 4096), (70, 200, 2048), (300, 520, 2048)])
def test_largest_sums_are_exact(gpu, m, n, k):
    """All codes +-127 with unit scales: sums far beyond 2^24, checked as the bf16 of the exact integer."""
    kp = (k + 127) // 128 * 128
    bufs = []
    for rows in (m, n):
        codes = torch.full((rows, k), 127, dtype=torch.int8)
        codes[::2] *= -1
        codes[:, ::3] -= torch.arange(rows, dtype=torch.int8)[:, None] * 0 + 1 * (codes[:, ::3] > 0)
        buf = torch.zeros(rows * (kp + 4), dtype=torch.uint8)
        buf[:rows * kp].view(torch.int8).view(rows, kp)[:, :k] = codes
        buf[rows * kp:].view(torch.float32).fill_(1.0)
        bufs.append((buf, codes, torch.ones(rows)))
    out = torch.zeros(m, n, dtype=torch.bfloat16, device=gpu)
    bq.w8a8_gemm(bufs[0][0].to(gpu), bufs[1][0].to(gpu), out, m, n, k)
    check_product(out.cpu(), bufs, None)


def test_nan_scale_stays_in_its_row_and_column(gpu):
    m, n, k = 5, 40, 256
    bufs, _ = product_case(m, n, k, 5)
    for buf, codes, scale in bufs:
        rows = len(scale)
        scale[2] = float("nan")
        buf[rows * 256:].view(torch.float32).copy_(scale)
    out = torch.zeros(m, n, dtype=torch.bfloat16, device=gpu)
    bq.w8a8_gemm(bufs[0][0].to(gpu), bufs[1][0].to(gpu), out, m, n, k)
    nan = out.cpu().isnan()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[2], want[:, 2] = True, True
    assert torch.equal(nan, want)


def test_norm_product_chain_on_another_stream_and_in_a_graph(gpu):
    """norm -> int8 rows -> product, eagerly, on a side stream and captured: the same bits each time; the graph is
    replayed with the program's own work and waits in between."""
    m, n, k = 37, 300, 1000
    x, r, w = (t.to(gpu) for t in make(m, k, 55))
    bufs, bias = product_case(m, n, k, 56)
    weight, bias = bufs[1][0].to(gpu), bias.to(gpu)

    def chain(r_, i8, out):
        bq.add_rms_norm_quantize_int8(x, r_, w, i8, m, k, EPS)
        bq.w8a8_gemm(i8, weight, out, m, n, k, bias=bias)

    def buffers():
        return (r.clone(), torch.zeros(bq.int8_rows_bytes(m, k), dtype=torch.uint8, device=gpu),
                torch.zeros(m, n, dtype=torch.bfloat16, device=gpu))

    eager = buffers()
    chain(*eager)
    side = buffers()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        chain(*side)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, side))
    got = buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(*got)
    for i in range(4):
        got[0].copy_(r)
        got[1].zero_()
        got[2].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, got)), i
