"""Every kernel that the int8 product can take, at one, two, three and more steps of k, with rows and columns left over,
against exact sums in 64 bits.  The form that a size takes is asked for, so that a change of the choice shows here.

Bounds, as in test_gpu_norm_w8a8: half a bf16 step, 2^-8 |y|, and four roundings in binary32 before it (the sum's
conversion, two scales, the bias), 2^-22 of |sum sa sw| + |bias|."""
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq

CUS = 256
CASES = [  # form, m, n, k
    (0, 1, 1, 1), (0, 16, 2000, 300), (0, 33, 40, 2563), (7, 2049, 3, 1), (7, 1, 2061, 129), (7, 16, 4099, 1000),
    (1, 50, 11458, 1), (1, 36, 10309, 129), (1, 33, 8155, 300), (1, 17, 9761, 1000),
    (2, 1181, 9857, 129), (2, 649, 11187, 300), (2, 65, 8749, 1500),
    (3, 1259, 9739, 200), (3, 4158, 1961, 300), (3, 4346, 403, 1500),
    (4, 3791, 4617, 1), (4, 916, 9826, 129), (4, 709, 11115, 300), (4, 259, 9955, 1000),
    (5, 3034, 4741, 1), (5, 585, 9870, 129), (5, 579, 9999, 500), (5, 652, 9129, 1000),
    (6, 31163, 18049, 100), (6, 28070, 9885, 200), (6, 7558, 25610, 300), (6, 4268, 10674, 1500),
    (8, 25667, 20097, 100), (8, 27006, 8579, 200), (8, 22676, 6535, 300), (8, 4353, 4097, 1030), (8, 1694, 10551, 1500),
]


def test_the_cases_reach_every_form():
    assert [bq.w8a8_gemm_form(*case[1:], CUS) for case in CASES] == [case[0] for case in CASES]
    assert {case[0] for case in CASES} == set(range(9))


def rows(n, k, gen, device):
    """int8 rows with every code, and scales that are no powers of two; the padding is zeros."""
    kp = (k + 127) // 128 * 128
    buf = torch.zeros(n * (kp + 4), dtype=torch.uint8, device=device)
    codes = buf[:n * kp].view(torch.int8).view(n, kp)[:, :k]
    codes.copy_(torch.randint(-127, 128, (n, k), generator=gen, device=device, dtype=torch.int8))
    scale = buf[n * kp:].view(torch.float32)
    scale.copy_(0.01 * torch.exp(torch.randn(n, generator=gen, device=device)))
    return buf, codes, scale


@pytest.mark.gpu
@pytest.mark.parametrize("form,m,n,k", CASES)
def test_form(gpu, form, m, n, k):
    print(f"w8a8 form {form} m={m} n={n} k={k}", flush=True)
    if torch.cuda.get_device_properties(gpu).multi_processor_count != CUS:
        pytest.skip("the forms are those of a whole card")
    gen = torch.Generator(device=gpu).manual_seed(m + n + k)
    act, a, sa = rows(m, k, gen, gpu)
    weight, w, sw = rows(n, k, gen, gpu)
    bias = torch.randn(n, generator=gen, device=gpu).bfloat16() if (m + n) % 2 else None
    out = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device=gpu)
    view = out[32:32 + m * n].view(m, n)
    bq.w8a8_gemm(act, weight, view, m, n, k, bias=bias)
    assert (out[:32] == 7).all() and (out[32 + m * n:] == 7).all()
    w = w.double().t().contiguous()
    for r in range(0, m, 4096):  # whole numbers below 2^31: exact in binary64
        p = (a[r:r + 4096].double() @ w) * sa[r:r + 4096, None].double() * sw.double()
        y = p if bias is None else p + bias.double()
        bound = 2.0 ** -8 * y.abs() + 2.0 ** -22 * (p.abs() + (0 if bias is None else bias.double().abs()))
        assert ((view[r:r + 4096].double() - y).abs() <= bound).all(), r
