"""The example block end to end: norm, int8 (and 2-bit) products, the delta rule in both forms, the FFN.

Bounds.  Against 64 bits without quantized activations: a row of int8 codes is off by a uniform error of step / sqrt(12)
with step = top / 127, which for normal rows (top about 4 times their root mean square) is 1% of the row.  Four products
follow each other and the delta rule multiplies q, k and v, each of which carries its 1%: 10%.  Where a head's o is
q.k of one token, its norm enlarges the error of a q.k near zero: with 1.4% of q.k's deviation off, 15% over normal q.k.
20% in all (a wrong operand, order or gate is off by about 100%).  Decoded tokens against one prefill: the int8 product does not depend on how rows
are batched, so the states differ by the two forms' own errors alone, twice 8 * 2^-24 * sqrt(T + 4) of their norm; the
outputs by bf16 steps that the int8 codes after them can turn into whole code steps, 1 / 127 of a row's largest value,
about 3% of its norm where every code is hit, and through two such products 6%."""
import os
import sys

import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from delta_ref import delta_reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from gated_delta_block import GatedDeltaBlock, prefill_and_decode  # noqa: E402

pytestmark = pytest.mark.gpu
SIZES = dict(hidden=256, hk=2, hv=4, dk=64, dv=64, ffn=384)


def int8_values(rows, n, k):
    rows, kp = rows.cpu(), (k + 127) // 128 * 128
    return (rows[:n * kp].view(torch.int8).view(n, kp)[:, :k].double()
            * rows[n * kp:n * (kp + 4)].view(torch.float32).double()[:, None])


def q2_0_values(w, n, k):
    w = w.cpu()
    groups = w[:n * k // 4].view(n, k // 128, 32)  # byte t of a group of 128: the codes of values t, t + 32, ...
    codes = torch.stack([groups >> s & 3 for s in (0, 2, 4, 6)], dim=2).view(n, k)
    return (codes.double() - 2) * w[n * k // 4:].view(torch.float16).double().view(n, k // 128).repeat_interleave(128, 1)


def norm(h, weight):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * weight.cpu().double()


def reference(block, x, residual, starts):
    hk, hv, dk, dv, hidden, ffn = block.hk, block.hv, block.dk, block.dv, block.hidden, block.ffn
    h = x.double() + residual.double()
    y = norm(h, block.norm1)
    w = (int8_values if block.qkvz == "int8" else q2_0_values)(block.w_qkvz, block.width, hidden)
    q, k, v, z = (y @ w.t()).split([hk * dk, hk * dk, hv * dv, hv * dv], dim=1)
    a, beta = (y @ int8_values(block.w_ab, 2 * hv, hidden).t()).split(hv, dim=1)
    g = -block.decay.cpu().double() * torch.nn.functional.softplus(a + block.bias.cpu().double())
    count = len(starts) - 1
    o, state, _ = delta_reference(q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv)), g,
                                  torch.sigmoid(beta), torch.zeros(count, hv, dk, dv), starts, None, None, True, dk ** -0.5)
    z = z * torch.sigmoid(z) * norm(o.flatten(0, 1), block.norm_o).view(z.shape)
    h = h + z @ int8_values(block.w_out, hidden, hv * dv).t()
    y = norm(h, block.norm2)
    gate, up = (y @ int8_values(w, ffn, hidden).t() for w in (block.w_gate, block.w_up))
    return (gate * torch.sigmoid(gate) * up) @ int8_values(block.w_down, hidden, ffn).t(), h, state


@pytest.mark.parametrize("qkvz", ["int8", "q2_0"])
def test_block_against_definition(gpu, qkvz):
    block = GatedDeltaBlock(**SIZES, qkvz=qkvz, device=gpu)
    starts = [0, 1, 71, 71, 200]
    gen = torch.Generator().manual_seed(3)
    x, residual = (torch.randn(200, 256, generator=gen).bfloat16() for _ in range(2))
    rd, state = residual.to(gpu), block.new_state(4)
    out = block(x.to(gpu), rd, state, torch.tensor(starts, dtype=torch.int32, device=gpu), None,
                torch.ones(4, dtype=torch.uint8, device=gpu), block.buffers(200, 4), prefill=True)
    for got, want in zip((out, rd, state), reference(block, x, residual, starts)):
        off = ((got.cpu().double() - want).norm() / want.norm()).item()
        assert off <= 0.2, off


@pytest.mark.parametrize("qkvz", ["int8", "q2_0"])
def test_decoded_tokens_continue_a_prefill(gpu, qkvz):
    block = GatedDeltaBlock(**SIZES, qkvz=qkvz, device=gpu)
    lens, steps = [70, 1, 130, 64], 4
    ends, decoded, whole, state = prefill_and_decode(block, lens, steps)
    assert (ends - decoded).float().norm() <= 0.06 * ends.float().norm()
    off = ((state - whole).double().norm() / whole.double().norm()).item()
    assert off <= 2 * 8 * 2.0 ** -24 * (max(lens) + steps + 4) ** 0.5, off
