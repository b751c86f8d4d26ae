"""The chunked gated delta rule where the workspace exceeds the caches and lines are touched ahead: what is touched
lies inside the tensors' own rows (a row expanded over all tokens ends with its last value), for short heads, and the
whole-head kernels of 64 and 128 with touching give what the definition says.  Bounds: those of test_gpu_delta_rule."""
import pytest
import torch

import bit_quantized_matmul_quantize_amd as bq
from test_gpu_delta_rule import call, check, heads, make

pytestmark = pytest.mark.gpu
TOUCHED = 128 << 20  # bytes of workspace beyond which lines are touched


def touches(d):
    return bq.gated_delta_rule_workspace_bytes(d["starts"][-1], len(d["starts"]) - 1, *d["sizes"]) > TOUCHED


@pytest.mark.parametrize("sizes", [(64, 64, 16, 64), (64, 64, 64, 16), (64, 64, 1, 1)], ids=lambda s: "x".join(map(str, s)))
def test_one_row_expanded_over_all_tokens(gpu, sizes):
    hk, hv, dk, dv = sizes
    tokens = 64 * 70 + 3
    d = make([tokens], *sizes, seed=61)
    assert touches(d)
    rows = [x[:1].contiguous().to(gpu) for x in (torch.randn(1, h, w, generator=torch.Generator().manual_seed(w)).bfloat16()
                                                 for h, w in ((hk, dk), (hk, dk), (hv, dv)))]
    g, beta = d["g"].to(gpu), d["beta"].to(gpu)
    starts = torch.tensor([0, tokens], dtype=torch.int32, device=gpu)
    work = torch.zeros(bq.gated_delta_rule_workspace_bytes(tokens, 1, *sizes), dtype=torch.uint8, device=gpu)
    results = []
    for copy in (False, True):
        qkv = [x.expand(tokens, *x.shape[1:]) for x in rows]
        assert all(x.stride(0) == 0 for x in qkv)
        if copy:
            qkv = [x.contiguous() for x in qkv]
        out, state = torch.zeros(tokens, hv, dv, dtype=torch.bfloat16, device=gpu), d["state"].to(gpu)
        bq.gated_delta_rule_chunked(*qkv, g, beta, out, state, starts, work, slots=d["slots"].to(gpu))
        results.append((out, state))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("sizes,lens", [((16, 32, 128, 128), [64 * 60 + 9, 64 * 45, 1, 130]), ((32, 64, 64, 64), [64 * 50, 64 * 12 + 1])],
                         ids=lambda s: "x".join(map(str, s)))
def test_whole_heads(gpu, sizes, lens):
    """All heads on the GPU; one key head's value heads against the definition (heads do not depend on each other)."""
    hk, hv, dk, dv = sizes
    d = make(lens, *sizes, seed=62)
    assert touches(d)
    fresh = [i % 2 for i in range(len(lens))]
    out, state = call(gpu, "chunked", d, fresh)
    assert out.isfinite().all() and state.isfinite().all()
    i, of = hk - 2, hv // hk
    q, k, v = heads(d, d["packed"])
    mine = slice(i * of, (i + 1) * of)
    one = {**d, "packed": torch.cat([q[:, i], k[:, i], v[:, mine].flatten(1)], dim=1), "g": d["g"][:, mine],
           "beta": d["beta"][:, mine], "state": d["state"][:, mine].contiguous(), "sizes": (1, of, dk, dv)}
    check(one, out[:, mine], state[:, mine].contiguous(), fresh)
