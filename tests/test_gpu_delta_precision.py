"""The gated delta rule's outputs are made from binary32: where large terms cancel, what is left is right.

Each test makes o as the difference of two nearly equal terms of size x that only a binary32 operand tells apart, in one
of the places where the chunked form has such operands: the state, U, and the decayed q.k triangle.  All other factors
are exact (zeros, ones, powers of two), so the roundings can be counted.

Bounds, with e = 2^-23 for a rounding in binary32 (twice the half step, as a matrix core may cut off): the two terms'
parts are added in at most 12 steps, none of which passes 2 x: 24 e x would be the worst of all, each of them rounding a
sum at its largest and the same way.  Of the 12 at most six parts of each term are not zero, and a term's second and
third parts are below 2^-8 x, so their sums among themselves do not count: 4 roundings of sums up to 2 x, 8 e x.  The
terms' own values: U = b v is off by e / 2, a decay by the power's last place and its argument's, 2 e, for each of two
terms and at most three decays in the recurrent form: 2 (e / 2 + 6 e) = 13 e.  Together below 2^-18 x (32 e), and half a
bf16 step of o, 2^-8 |o|.  Operands of two bf16 parts (2^-16) would be off by up to 2^-15 x."""
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq

pytestmark = pytest.mark.gpu
FORMS = ["recurrent", "chunked"]


def run(gpu, form, q, k, v, g, beta, state):
    tokens, hk, dk = q.shape
    hv, dv = v.shape[1:]
    out = torch.full((tokens, hv, dv), 7.0, dtype=torch.bfloat16, device=gpu)
    state = state.to(gpu)
    args = (*(x.bfloat16().to(gpu) for x in (q, k, v)), g.to(gpu), beta.to(gpu), out, state,
            torch.tensor([0, tokens], dtype=torch.int32, device=gpu))
    if form == "recurrent":
        bq.gated_delta_rule_recurrent(*args, l2norm=False, scale=1.0)
    else:
        work = torch.zeros(bq.gated_delta_rule_workspace_bytes(tokens, 1, hk, hv, dk, dv), dtype=torch.uint8, device=gpu)
        bq.gated_delta_rule_chunked(*args, work, l2norm=False, scale=1.0)
    return out.cpu().double(), state.cpu()


def check(out, want, x):
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -18 * x.abs()
    off = (out - want).abs()
    assert (want.abs() < 2.0 ** -9 * x.abs()).double().mean() > 0.9  # the terms do cancel
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens,hv,dk,dv", [(130, 2, 128, 64), (130, 2, 64, 64), (70, 1, 100, 33), (2100, 1, 128, 32),
                                             (2100, 1, 64, 32)])
def test_state(gpu, form, tokens, hv, dk, dv):
    """Nothing is written (beta = 0) or forgotten: o_t = S_i - S_j, rows that agree to 2^-12."""
    gen = torch.Generator().manual_seed(41 + dk + tokens)
    state = torch.randn(1, hv, dk, dv, generator=gen)
    state[:, :, 1::2] = state[:, :, ::2] * (1 + 2.0 ** -12 * torch.randn(1, hv, dk // 2, dv, generator=gen))
    q, row = torch.zeros(tokens, 1, dk), torch.arange(tokens) % (dk // 2) * 2
    q[torch.arange(tokens), 0, row], q[torch.arange(tokens), 0, row + 1] = 1.0, -1.0
    k, v = torch.randn(tokens, 1, dk, generator=gen), torch.randn(tokens, hv, dv, generator=gen)
    g = beta = torch.zeros(tokens, hv)
    out, after = run(gpu, form, q, k, v, g, beta, state)
    assert torch.equal(after, state)
    a, b = state[0, :, row].transpose(0, 1).double(), state[0, :, row + 1].transpose(0, 1).double()
    check(out, a - b, a)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 64), (100, 33)])
def test_within_a_chunk(gpu, form, decay, dk, dv):
    """Keys of their own axes from an empty state, so u_t = beta_t v; q_t takes the two tokens before it, whose betas
    (with the decay between them) agree to 2^-12."""
    tokens, hv = 64, 2
    gen = torch.Generator().manual_seed(51 + dk)
    k = torch.zeros(tokens, 1, dk)
    k[torch.arange(tokens), 0, torch.arange(tokens)] = 1.0
    q = torch.zeros(tokens, 1, dk)
    t = torch.arange(2, tokens)
    q[t, 0, t - 2], q[t, 0, t - 1] = 1.0, -1.0
    v = torch.randn(1, hv, dv, generator=gen).bfloat16().expand(tokens, hv, dv)
    g = -0.05 * torch.rand(tokens, hv, generator=gen) if decay else torch.zeros(tokens, hv)
    beta = torch.empty(tokens, hv)
    beta[0] = 0.9
    for i in range(1, tokens):  # what is left of the token before, and a little more or less
        beta[i] = (beta[i - 1].double() * torch.exp(g[i].double()) * (1 + 2.0 ** -12 * torch.randn(hv, generator=gen))).float()
    out, _ = run(gpu, form, q, k, v, g, beta, torch.zeros(1, hv, dk, dv))
    u, e = beta.double()[:, :, None] * v.double(), torch.exp(g.double())[:, :, None]
    one, two = e[2:] * e[1:-1] * u[:-2], e[2:] * u[1:-1]
    check(out[2:], one - two, one)
