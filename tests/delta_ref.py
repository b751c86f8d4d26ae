"""The gated delta rule in 64 bits on the CPU, token by token, for the GPU tests.

Per value head, a = exp(g), b = beta:  S = a S;  S = S + k (b (v - k^T S))^T;  o = scale q^T S."""
import torch


def delta_reference(q, k, v, g, beta, state, starts, slots, fresh, l2norm, scale, dtype=torch.float64):
    """Returns (out, state, largest column norm of S so far at each token).  Everything on the CPU; sequences with a
    slot outside the state start from zeros and are not kept."""
    q, k, v, g, beta = (x.to(dtype) for x in (q, k, v, g, beta))
    state = state.to(dtype).clone()
    hv, hk = v.shape[1], q.shape[1]
    if l2norm:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = (x.repeat_interleave(hv // hk, 1) for x in (q, k))
    out = torch.full(v.shape, float("nan"), dtype=dtype)
    top = torch.zeros(v.shape, dtype=dtype)
    for i in range(len(starts) - 1):
        slot = i if slots is None else slots[i]
        kept = 0 <= slot < state.shape[0]
        new = not kept or (fresh is not None and bool(fresh[i]))
        S = torch.zeros(hv, q.shape[2], v.shape[2], dtype=dtype) if new else state[slot].clone()
        most = S.norm(dim=1)
        for t in range(starts[i], starts[i + 1]):
            S = S * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
            S = S + k[t][:, :, None] * u[:, None, :]
            out[t] = scale * (q[t][:, :, None] * S).sum(1)
            most = torch.maximum(most, S.norm(dim=1))
            top[t] = most
        if kept:
            state[slot] = S
    return out, state, top
