"""The example block with buffers that were made for more tokens and prompts than a call has, as a server keeps them."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from gated_delta_block import GatedDeltaBlock  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qkvz", ["int8", "q2_0"])
@pytest.mark.parametrize("starts", [[0, 130], [0, 1, 71, 71, 200], [0, 40, 41]], ids=str)
def test_buffers_of_up_to_so_many_tokens(gpu, qkvz, starts):
    block = GatedDeltaBlock(hidden=256, hk=2, hv=4, dk=64, dv=64, ffn=384, qkvz=qkvz, device=gpu)
    count, m = len(starts) - 1, starts[-1]
    gen = torch.Generator().manual_seed(m)
    x, residual = (torch.randn(m, 256, generator=gen).bfloat16().to(gpu) for _ in range(2))
    got = []
    for prefill in (True, False):
        for b in (block.buffers(m, count), block.buffers(200, 4)):
            for t in b.values():
                t.view(torch.uint8).fill_(0xFF)  # NaN in every bf16
            state, r = block.new_state(count), residual.clone()
            out = block(x, r, state, torch.tensor(starts, dtype=torch.int32, device=gpu), None,
                        torch.ones(count, dtype=torch.uint8, device=gpu), b, prefill)
            assert out.shape == x.shape
            got.append([t.cpu() for t in (out, r, state)])
    assert all(torch.equal(s, t) for s, t in zip(got[0], got[1]))
    assert all(torch.equal(s, t) for s, t in zip(got[2], got[3]))
    assert all(t.isfinite().all() for t in got[1])
