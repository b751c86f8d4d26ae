"""The paged key-value cache and the attention over it in 64 bits on the CPU, for the GPU tests.

A page holds, for each key head, a block of page * d values in units of 16 bytes (U = 8 bf16 values or 16 int8 codes),
and behind int8 codes a binary32 scale for each token.  Value j of token o: keys at ((j / U) P + o) U + j % U, values at
((o / U) d + j) U + o % U."""
import numpy as np
import torch


def block_bytes(page, d, bits):
    return 2 * page * d if bits == 16 else page * (d + 4)


def places(page, d, bits, keys):
    """Index within a block of each [token, value] of a page."""
    unit = 8 if bits == 16 else 16
    o, j = np.arange(page)[:, None], np.arange(d)[None, :]
    return ((j // unit) * page + o) * unit + j % unit if keys else ((o // unit) * d + j) * unit + o % unit


class Cache:
    """A pool of pages in host memory, every byte 0xFF (a NaN as bf16 and as a scale) until it is written."""

    def __init__(self, pages, page, hk, d, bits):
        self.pages, self.page, self.hk, self.d, self.bits = pages, page, hk, d, bits
        self.block = block_bytes(page, d, bits)
        self.k = np.full(pages * hk * self.block, 0xFF, dtype=np.uint8)
        self.v = self.k.copy()

    def _at(self, keys, page_id, head):
        b = (self.k if keys else self.v).reshape(self.pages, self.hk, self.block)[page_id, head]
        return b, places(self.page, self.d, self.bits, keys)

    def put(self, keys, page_id, o, rows):
        """rows: [hk, d], bf16 values in float64 (bits 16), or (codes [hk, d], scales [hk])."""
        for h in range(self.hk):
            b, at = self._at(keys, page_id, h)
            if self.bits == 16:
                b.view(np.uint16)[at[o]] = torch.from_numpy(rows[h]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
            else:
                b[:self.page * self.d].view(np.int8)[at[o]] = rows[0][h]
                b[self.page * self.d:].view(np.float32)[o] = rows[1][h]

    def get(self, keys, page_id, o):
        """[hk, d] in float64."""
        out = np.empty((self.hk, self.d))
        for h in range(self.hk):
            b, at = self._at(keys, page_id, h)
            if self.bits == 16:
                out[h] = torch.from_numpy(b.view(np.int16)[at[o]].copy()).view(torch.bfloat16).double().numpy()
            else:
                out[h] = b[:self.page * self.d].view(np.int8)[at[o]].astype(np.float64) * float(b[self.page * self.d:].view(np.float32)[o])
        return out


class Case:
    """Packed sequences over a cache: lens is a list of (new tokens, all tokens); pages in no order, entries of the
    table behind a sequence's last page outside the pool."""

    def __init__(self, lens, hq, hk, d, bits, page, seed, spread=1.0, extra=16):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hk, self.d, self.bits, self.page = lens, hq, hk, d, bits, page
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.tokens = int(self.starts[-1])
        used = [-(-total // page) for _, total in lens]
        pages = sum(used) + 2
        width = max(max(used, default=1), 1) + 1
        order = torch.randperm(pages, generator=gen).numpy()
        self.table = np.full((len(lens), width), -1, dtype=np.int32)
        self.table[:, -1] = 1 << 30
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.cache = Cache(pages, page, hk, d, bits)
        self.rows = []
        for i, (_, total) in enumerate(lens):
            pair = []
            for keys in (True, False):
                x = (spread if keys else 1.0) * torch.randn(total, hk, d, generator=gen)
                if bits == 16:
                    x = x.bfloat16().double().numpy()
                    for p in range(total):
                        self.cache.put(keys, self.table[i, p // page], p % page, x[p])
                else:
                    codes = torch.randint(-127, 128, (total, hk, d), generator=gen).numpy()
                    scales = ((0.5 + torch.rand(total, hk, generator=gen)) / 60 * (spread if keys else 1.0)).float().numpy()
                    for p in range(total):
                        self.cache.put(keys, self.table[i, p // page], p % page, (codes[p], scales[p]))
                    x = codes * scales.astype(np.float64)[:, :, None]
                pair.append(x)
            self.rows.append(pair)
        self.packed = torch.randn(self.tokens, hq * d + extra, generator=gen).bfloat16()

    def device(self, gpu):
        def t(x):
            return torch.from_numpy(np.ascontiguousarray(x)).to(gpu)
        return dict(q=self.packed.to(gpu)[:, :self.hq * self.d].unflatten(1, (self.hq, self.d)), k_cache=t(self.cache.k),
                    v_cache=t(self.cache.v), starts=t(self.starts), lens=t(np.array([n for _, n in self.lens], dtype=np.int32)),
                    table=t(self.table))

    def q(self):
        return self.packed[:, :self.hq * self.d].double().numpy().reshape(self.tokens, self.hq, self.d)


def attention(case, window=0, cap=0.0, scale=None):
    """(out, sum_j p_j |v_j| / sum_j p_j, largest scale |q| . |k_j| that is seen), [tokens, hq, d] and [tokens, hq, 1]."""
    scale = case.d ** -0.5 if scale is None else scale
    g = case.hq // case.hk
    q = case.q()
    out, size = np.zeros((2, case.tokens, case.hq, case.d))
    most = np.zeros((case.tokens, case.hq, 1))
    for i, (n, total) in enumerate(case.lens):
        s0 = int(case.starts[i])
        k, v = case.rows[i]
        for t in range(n):
            p = total - n + t
            lo = max(0, p + 1 - window) if window else 0
            for h in range(case.hq):
                kk, vv = k[lo:p + 1, h // g], v[lo:p + 1, h // g]
                s = scale * (kk @ q[s0 + t, h])
                most[s0 + t, h] = (scale * (np.abs(kk) @ np.abs(q[s0 + t, h]))).max()
                if cap:
                    s = cap * np.tanh(s / cap)
                w = np.exp(s - s.max())
                out[s0 + t, h] = w @ vv / w.sum()
                size[s0 + t, h] = w @ np.abs(vv) / w.sum()
    return out, size, most


def bound(case, out, size, most, form, cap=0.0):
    """How far an output may be off: half a step of bf16, 2^-8 of it, and of sum p |v| / sum p:
    - the weights' rounding: 2^-16 as sums of two bf16 (the rest of the first is rounded by 2^-8 of 2^-8), 2^-8 as one;
      as one the sum may be that of the rounded weights w (1 + e): sum w e (v - out) / sum w, 2^-8 of |out| more;
    - the score's error: d products summed in binary32 and a few roundings, (d + 8) 2^-24 of scale |q| . |k|, and under a
      cap 2^-21 of the cap (a hardware exponential and reciprocal); a weight moves by as much relative to itself, and the
      sum of the weights too: twice;
    - the hardware's exp2 and the sums of the weights, 2^-20 (a sum of up to 2^16 positive terms in chains of a lane's);
    - weights and products below 2^-126 may be flushed to zero (binary32's and bf16's normal range ends there): 2^16 keys
      of values up to 2^8 lose at most 2^(16 + 8 - 126) < 2^-100."""
    score = (case.d + 8) * 2.0 ** -24 * most + (2.0 ** -21 * cap if cap else 0.0)
    weight = 2.0 ** -16 if form == "decode" else 2.0 ** -8
    halves = 1 if form == "decode" else 2
    return halves * 2.0 ** -8 * np.abs(out) + size * (weight + 2 * score + 2.0 ** -14) * (1 + 2.0 ** -8) + 2.0 ** -100


def rope(x, cos_sin, rows, norm, eps):
    """x: [tokens, heads, d]; rows: [tokens, rot / 2] row of cos_sin of each frequency.  Also the sizes of the terms."""
    d, half = x.shape[-1], rows.shape[1]
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm
    f = np.arange(half)
    c, s = cos_sin[rows, 0, f][:, None, :], cos_sin[rows, 1, f][:, None, :]
    a, b = x[..., :half], x[..., half:2 * half]
    y, size = x.copy(), np.abs(x)
    y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    size[..., :half] = np.abs(a * c) + np.abs(b * s)
    size[..., half:2 * half] = np.abs(b * c) + np.abs(a * s)
    return y, size


def table_of_angles(angles, rot, theta=1e6):
    a = np.arange(angles)[:, None] * theta ** (-np.arange(rot // 2) / max(1, rot // 2))
    return np.stack([np.cos(a), np.sin(a)], 1).astype(np.float32)


__all__ = ["Cache", "Case", "attention", "block_bytes", "bound", "places", "rope", "table_of_angles"]
