"""A block of a gated-delta-rule model served through the package: prompts of ragged lengths in one packed batch,
then decoded tokens of the same sequences.

    residual += x;  y = norm(residual)                       add_rms_norm_quantize_int8 / _q8_1
    q | k | v | z = y Wqkvz^T,  a | b = y Wab^T                w8a8_gemm (or q2_0_mmq_gemm for a 2-bit Wqkvz)
    g = -A softplus(a + bias),  beta = sigmoid(b)
    o = delta rule of q, k, v, g, beta and the state         gated_delta_rule_chunked / _recurrent
    x = (silu(z) norm(o)) Wout^T, the norm per head          add_rms_norm_bf16, silu_mul_bf16, quantize_rows_int8, w8a8_gemm
    residual += x;  y = norm(residual)                       add_rms_norm_quantize_int8
    x = (silu(y Wgate^T) (y Wup^T)) Wdown^T                  w8a8_gemm, silu_mul_bf16, quantize_rows_int8

The sizes are those of the projections that the package is measured on (hidden 2048, 16 key and 32 value heads of
128, so that Wqkvz has 12288 rows); the weights are random.  Run it on a GPU: it prints the time of a prefill and of
a decode step (eager, and replayed from a graph), and how far the decoded tokens are from one prefill over all of
them.

    python examples/gated_delta_block.py [--qkvz q2_0]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_matmul_quantize_amd as bq  # noqa: E402


def int8_weight(w):
    """bf16 [n, k] as int8 rows."""
    n, k = w.shape
    rows = torch.empty(bq.int8_rows_bytes(n, k), dtype=torch.uint8, device=w.device)
    bq.quantize_rows_int8(w.bfloat16().contiguous(), rows, n, k)
    return rows


def random_q2_0(n, k, gen, device):
    """Random 2-bit codes with scales near the standard deviation 0.02 of the other weights."""
    codes = torch.randint(0, 256, (n * k // 4,), generator=gen, device=device, dtype=torch.uint8)
    scales = (0.02 * torch.rand(n * k // 128, generator=gen, device=device)).half()
    return torch.cat([codes, scales.view(torch.uint8)])


class GatedDeltaBlock:
    def __init__(self, hidden=2048, hk=16, hv=32, dk=128, dv=128, ffn=5120, qkvz="int8", device="cuda", seed=0):
        self.hidden, self.hk, self.hv, self.dk, self.dv, self.ffn, self.qkvz = hidden, hk, hv, dk, dv, ffn, qkvz
        self.width = 2 * hk * dk + 2 * hv * dv  # of a row of q | k | v | z
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return int8_weight(0.02 * torch.randn(n, k, generator=gen, device=device))

        self.w_qkvz = weight(self.width, hidden) if qkvz == "int8" else random_q2_0(self.width, hidden, gen, device)
        self.w_ab, self.w_out = weight(2 * hv, hidden), weight(hidden, hv * dv)
        self.w_gate, self.w_up, self.w_down = weight(ffn, hidden), weight(ffn, hidden), weight(hidden, ffn)
        self.norm1 = (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).bfloat16()
        self.norm2 = (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).bfloat16()
        self.norm_o = (1 + 0.1 * torch.randn(dv, generator=gen, device=device)).bfloat16()
        self.decay = 0.5 + 15.5 * torch.rand(hv, generator=gen, device=device)
        self.bias = torch.randn(hv, generator=gen, device=device) - 4.0
        self.device = device

    def new_state(self, slots):
        return torch.zeros(slots, self.hv, self.dk, self.dv, device=self.device)

    def buffers(self, tokens, count=0):
        """What a call of up to `tokens` tokens writes on its way; count: the prompts of a prefill."""
        def bf(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=self.device)

        def u8(size):
            return torch.empty(size, dtype=torch.uint8, device=self.device)

        b = dict(norm=u8(bq.int8_rows_bytes(tokens, self.hidden)), qkvz=bf(tokens, self.width), ab=bf(tokens, 2 * self.hv),
                 o=bf(tokens, self.hv, self.dv), normed=bf(tokens, self.hv * self.dv), gated=u8(bq.int8_rows_bytes(tokens, self.hv * self.dv)),
                 gate=bf(tokens, self.ffn), up=bf(tokens, self.ffn), wide=u8(bq.int8_rows_bytes(tokens, self.ffn)),
                 out=bf(tokens, self.hidden))
        if self.qkvz == "q2_0":
            b["q8"] = u8(bq.q8_1_act_bytes(tokens, self.hidden))
        if count:
            b["workspace"] = u8(bq.gated_delta_rule_workspace_bytes(tokens, count, self.hk, self.hv, self.dk, self.dv))
        return b

    def __call__(self, x, residual, state, starts, slots, fresh, b, prefill):
        """x, residual: [tokens, hidden] bf16, the residual is updated in place; returns the block's x."""
        m, hidden, hk, hv, dk, dv = x.shape[0], self.hidden, self.hk, self.hv, self.dk, self.dv
        b = {name: t[:m] if t.dim() > 1 else t for name, t in b.items()}  # (they may be for more tokens)
        if self.qkvz == "q2_0":
            # both formats of the normalised rows; the second pass finds the sum in the residual
            bq.add_rms_norm_quantize_int8(x, residual, self.norm1, b["norm"], m, hidden)
            bq.add_rms_norm_quantize_q8_1(residual, None, self.norm1, b["q8"], m, hidden)
            bq.q2_0_mmq_gemm(b["q8"], self.w_qkvz, b["qkvz"], m, self.width, hidden)
        else:
            bq.add_rms_norm_quantize_int8(x, residual, self.norm1, b["norm"], m, hidden)
            bq.w8a8_gemm(b["norm"], self.w_qkvz, b["qkvz"], m, self.width, hidden)
        bq.w8a8_gemm(b["norm"], self.w_ab, b["ab"], m, 2 * hv, hidden)
        a, beta = b["ab"].float().split(hv, dim=1)
        g = -self.decay * torch.nn.functional.softplus(a + self.bias)
        beta = torch.sigmoid(beta)

        q, k, v, z = b["qkvz"].split([hk * dk, hk * dk, hv * dv, hv * dv], dim=1)
        args = (q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv)), g, beta, b["o"], state, starts)
        if prefill:
            bq.gated_delta_rule_chunked(*args, b["workspace"], slots=slots, fresh=fresh)
        else:
            bq.gated_delta_rule_recurrent(*args, slots=slots, fresh=fresh)
        bq.add_rms_norm_bf16(b["o"], None, self.norm_o, b["normed"], m * hv, dv)
        z = z.contiguous()
        bq.silu_mul_bf16(z, b["normed"], z)
        bq.quantize_rows_int8(z, b["gated"], m, hv * dv)
        bq.w8a8_gemm(b["gated"], self.w_out, b["out"], m, hidden, hv * dv)

        bq.add_rms_norm_quantize_int8(b["out"], residual, self.norm2, b["norm"], m, hidden)
        bq.w8a8_gemm(b["norm"], self.w_gate, b["gate"], m, self.ffn, hidden)
        bq.w8a8_gemm(b["norm"], self.w_up, b["up"], m, self.ffn, hidden)
        bq.silu_mul_bf16(b["gate"], b["up"], b["gate"])
        bq.quantize_rows_int8(b["gate"], b["wide"], m, self.ffn)
        bq.w8a8_gemm(b["wide"], self.w_down, b["out"], m, hidden, self.ffn)
        return b["out"]


def prefill_and_decode(block, lens, steps, seed=1):
    """Prompts of these lengths and then `steps` tokens each, against one prefill over all of it.  Returns the last
    tokens' outputs of both ways, [sequences, steps, hidden], and the states."""
    count, dev = len(lens), block.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows = [torch.randn(n + steps, block.hidden, generator=gen, device=dev).bfloat16() for n in lens]
    slots = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    fresh = torch.ones(count, dtype=torch.uint8, device=dev)

    def starts(sizes):
        return torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device=dev)

    def prefill(sizes, state):
        x = torch.cat([r[:n] for r, n in zip(rows, sizes)])
        b = block.buffers(x.shape[0], count)
        return block(x, torch.zeros_like(x), state, starts(sizes), slots, fresh, b, prefill=True).clone()

    whole = block.new_state(count)
    out = prefill([n + steps for n in lens], whole)
    ends = [o[-steps:] for o in out.split([n + steps for n in lens])]

    state = block.new_state(count)
    prefill(lens, state)
    b, one_each = block.buffers(count), starts([1] * count)
    decoded = []
    for t in range(steps):
        x = torch.stack([r[n + t] for r, n in zip(rows, lens)])
        decoded.append(block(x, torch.zeros_like(x), state, one_each, slots, None, b, prefill=False).clone())
    return torch.stack(ends), torch.stack(decoded, dim=1), whole, state


def timed(run, times=20):
    run()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(times):
        run()
    torch.cuda.synchronize()
    return (time.perf_counter() - t0) / times * 1e3


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--qkvz", choices=["int8", "q2_0"], default="int8")
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--batch", type=int, default=16)
    args = p.parse_args()
    block = GatedDeltaBlock(qkvz=args.qkvz)

    one, two, whole, state = prefill_and_decode(block, [70, 1, 300, 64], 6)
    print("decoded tokens against one prefill: outputs off by %.2e of their norm, states by %.2e" %
          (((one - two).float().norm() / one.float().norm()).item(), ((whole - state).norm() / whole.norm()).item()))

    x = torch.randn(args.tokens, block.hidden, device="cuda").bfloat16()
    residual, state = torch.zeros_like(x), block.new_state(args.batch)
    slots = torch.arange(args.batch, dtype=torch.int32, device="cuda")
    fresh = torch.ones(1, dtype=torch.uint8, device="cuda")
    starts, b = torch.tensor([0, args.tokens], dtype=torch.int32, device="cuda"), block.buffers(args.tokens, 1)
    print("prefill of %d tokens: %.3f ms" % (args.tokens, timed(
        lambda: block(x, residual.zero_(), state, starts, slots[:1], fresh, b, prefill=True))))

    x, residual = x[:args.batch].clone(), torch.zeros(args.batch, block.hidden, dtype=torch.bfloat16, device="cuda")
    each, b = torch.arange(args.batch + 1, dtype=torch.int32, device="cuda"), block.buffers(args.batch)

    def step():
        return block(x, residual.zero_(), state, each, slots, None, b, prefill=False)

    print("decode step of %d sequences: %.3f ms" % (args.batch, timed(step)), end="")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    print(", from a graph %.3f ms" % timed(graph.replay))


if __name__ == "__main__":
    main()
