"""Host-side refusals (no GPU) of the paged cache and its attention: the C ABI's argument checks, which run before any
HIP call, and the binding's checks of types, shapes and sizes; the layout's sizes."""
import ctypes

import pytest
import torch

from paged_ref import block_bytes


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


NAMES = {
    "rope_write_kv_cache": dict(
        q=at(1), k=at(2), v=at(3), q_out=at(4), k_cache=at(5), v_cache=at(6), starts=at(7), lens=at(8), table=at(9),
        cos_sin=at(10), positions=at(11), axis=at(12), q_norm=at(13), k_norm=at(14), tokens=8, count=2, pages=10, page=16,
        width=4, bits=16, hq=4, hk=2, d=64, rot=64, angles=100, axes=3, q_token=512, q_head=64, k_token=512, k_head=64,
        v_token=512, v_head=64, eps=1e-6, stream=None),
    "read_kv_cache": dict(
        k_cache=at(5), v_cache=at(6), k=at(2), v=at(3), starts=at(7), lens=at(8), table=at(9), tokens=8, count=2, pages=10,
        page=16, width=4, bits=16, hk=2, d=64, stream=None),
    "paged_attention_decode": dict(
        q=at(1), k_cache=at(5), v_cache=at(6), out=at(4), starts=at(7), lens=at(8), table=at(9), workspace=at(15),
        workspace_bytes=1 << 27, tokens=8, count=2, pages=10, page=16, width=4, bits=16, hq=4, hk=2, d=64, q_token=256,
        q_head=64, window=0, scale=0.125, cap=0.0, stream=None),
    "paged_attention_prefill": dict(
        q=at(1), k_cache=at(5), v_cache=at(6), out=at(4), starts=at(7), lens=at(8), table=at(9), tokens=8, count=2, pages=10,
        page=16, width=4, bits=16, hq=4, hk=2, d=64, q_token=256, q_head=64, window=0, scale=0.125, cap=0.0, stream=None),
}
ALL = list(NAMES)
ATTENTION = ["paged_attention_decode", "paged_attention_prefill"]
WRITE = ["rope_write_kv_cache"]


def refused(bq, name, status, needle, **change):
    args = {**NAMES[name], **change}
    assert len(args) == len(NAMES[name])
    assert getattr(bq.lib(), name)(*args.values()) == status, bq.lib().bq_last_error()
    assert needle in bq.lib().bq_last_error().decode()


@pytest.mark.parametrize("names,status,needle,change", [
    (ALL, -1, "null", dict(k_cache=None)),
    (ALL, -1, "null", dict(starts=None)),
    (ALL, -1, "null", dict(lens=None)),
    (ALL, -1, "null", dict(table=None)),
    (ALL, -2, "bits=4", dict(bits=4)),
    (ALL, -2, "page=8", dict(page=8)),
    (ALL, -2, "page=48", dict(page=48)),
    (ALL, -2, "page=2048", dict(page=2048)),
    (ALL, -2, "d=72", dict(d=72)),
    (ALL, -2, "d=0", dict(d=0)),
    (ALL, -2, "d=272", dict(d=272)),
    (ALL, -1, "hk=0", dict(hk=0)),
    (ALL, -1, "hk=65536", dict(hk=65536)),
    (ALL, -1, "pages=0", dict(pages=0)),
    (ALL, -1, "width=0", dict(width=0)),
    (ALL, -1, "width", dict(width=(1 << 26) + 1)),
    (ALL, -1, "too large", dict(tokens=(1 << 30) + 1)),
    (ALL, -1, "too large", dict(tokens=1 << 29, count=1 << 29)),
    (ALL, -3, "aligned", dict(k_cache=P(0x50000008))),
    (ALL, -3, "aligned", dict(table=P(0x90000002))),
    (WRITE, -1, "null", dict(k=None)),
    (WRITE, -1, "null", dict(q=None)),
    (WRITE, -1, "null", dict(q_out=None)),
    (WRITE, -1, "null", dict(cos_sin=None)),
    (WRITE, -1, "null", dict(angles=0)),
    (WRITE, -2, "rot=24", dict(rot=24)),
    (WRITE, -2, "rot=80", dict(rot=80)),
    (WRITE, -1, "eps", dict(eps=float("nan"))),
    (WRITE, -1, "axes", dict(axes=0)),
    (WRITE, -1, "axes", dict(axes=256)),
    (WRITE, -1, "without positions", dict(positions=None)),
    (WRITE, -1, "strides of k", dict(k_token=1 << 31)),
    (WRITE, -3, "heads of q", dict(q_head=68)),
    (WRITE, -3, "heads of v", dict(v=P(0x30000004))),
    (WRITE, -3, "output", dict(q_out=P(0x40000008))),
    (WRITE, -3, "norms", dict(k_norm=P(0xE0000002))),
    (WRITE, -1, "the output overlaps q", dict(q_out=P(0x10000100))),
    (WRITE, -1, "the output overlaps the keys' cache", dict(q_out=P(0x50000100))),
    (WRITE, -1, "the keys' cache overlaps k", dict(k_cache=P(0x20000100))),
    (WRITE, -1, "the values' cache overlaps the table", dict(v_cache=P(0x90000000))),
    (WRITE, -1, "the caches overlap", dict(v_cache=P(0x50000100))),
    (["read_kv_cache"], -1, "null", dict(v=None)),
    (["read_kv_cache"], -3, "aligned", dict(v=P(0x30000008))),
    (["read_kv_cache"], -1, "k overlaps v", dict(v=P(0x20000100))),
    (["read_kv_cache"], -1, "v overlaps the values' cache", dict(v=P(0x60000000))),
    (ATTENTION, -1, "null", dict(q=None)),
    (ATTENTION, -1, "null", dict(out=None)),
    (ATTENTION, -1, "divide", dict(hq=5)),
    (ATTENTION, -1, "divide", dict(hq=0)),
    (ATTENTION, -1, "scale", dict(scale=-1.0)),
    (ATTENTION, -1, "scale", dict(scale=float("nan"))),
    (ATTENTION, -1, "cap", dict(cap=-1.0)),
    (ATTENTION, -1, "cap", dict(cap=float("nan"))),
    (ATTENTION, -1, "window", dict(window=(1 << 30) + 1)),
    (ATTENTION, -1, "too large", dict(tokens=1 << 22)),
    (ATTENTION, -3, "heads of q", dict(q_token=260)),
    (ATTENTION, -3, "output", dict(out=P(0x40000008))),
    (ATTENTION, -1, "the output overlaps q", dict(out=P(0x10000100))),
    (ATTENTION, -1, "the output overlaps the keys' cache", dict(out=P(0x50000100))),
    (ATTENTION, -1, "the output overlaps lens", dict(out=P(0x80000000))),
    (ATTENTION[:1], -1, "null workspace", dict(workspace=None)),
    (ATTENTION[:1], -1, "needed", dict(workspace_bytes=1000)),
    (ATTENTION[:1], -3, "workspace", dict(workspace=P(0xF0000008))),
    (ATTENTION[:1], -1, "the workspace overlaps the output", dict(workspace=P(0x40000000 - 4096))),
])
def test_refusals(bq, names, status, needle, change):
    for name in names:
        refused(bq, name, status, needle, **change)


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("change", [dict(tokens=0), dict(count=0)])
def test_nothing_to_do(bq, name, change):
    args = {k: None if isinstance(v, P) else v for k, v in {**NAMES[name], **change}.items()}
    if "axis" in args:
        args["axes"] = 1
    assert getattr(bq.lib(), name)(*args.values()) == 0


def test_sizes(bq):
    for page in (16, 64, 1024):
        for hk, d in ((1, 16), (8, 128), (2, 256)):
            for bits in (16, 8):
                assert bq.kv_cache_page_bytes(page, hk, d, bits) == hk * block_bytes(page, d, bits)
    for bad in ((17, 1, 64, 16), (16, 0, 64, 16), (16, 1, 65, 16), (16, 1, 64, 4), (16, 1, 272, 8)):
        assert bq.kv_cache_page_bytes(*bad) == 0
    for bad in ((1, 1, 3, 2, 64), (1, 1, 0, 1, 64), (1, 1, 2, 2, 65), (1 << 24, 1, 2, 2, 64)):
        assert bq.paged_attention_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (16, 2, 256), (12, 12, 80), (24, 1, 64), (3, 3, 16), (70, 1, 256)])
def test_a_workspace_serves_smaller_calls(bq, hq, hk, d):
    # a call is refused one byte below what it needs; what it needs is at most the size asked for any larger call
    name = "paged_attention_decode"

    def fits(size, tokens, count):
        args = {**NAMES[name], "hq": hq, "hk": hk, "d": d, "tokens": tokens, "count": count, "workspace_bytes": size,
                "out": at(1)}  # (overlaps q: refused in any case, for the size where that is too small)
        bq.lib().paged_attention_decode(*{**args, "workspace": at(1), "out": at(200), "q_token": hq * d, "q_head": d}.values())
        return "needed" not in bq.lib().bq_last_error().decode()

    assert not fits(0, 1, 1)
    for tokens in (1, 2, 3, 5, 17, 64, 100):
        for count in (1, 2, 7, 50, 100, 300):
            size = bq.paged_attention_workspace_bytes(tokens, count, hq, hk, d)
            for t in (1, 2, 4, 16, 33, 64, 100):
                for c in (1, 2, 5, 31, 64, 100, 300):
                    if t <= tokens and c <= count:
                        assert fits(size, t, c), (tokens, count, t, c)


def tensors(**change):
    t = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k=torch.zeros(3, 2, 64, dtype=torch.bfloat16),
             v=torch.zeros(3, 2, 64, dtype=torch.bfloat16), out=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
             k_cache=torch.zeros(8192 * 5, dtype=torch.uint8), v_cache=torch.zeros(8192 * 5, dtype=torch.uint8),
             starts=torch.zeros(3, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32),
             table=torch.zeros(2, 4, dtype=torch.int32), workspace=torch.zeros(100, dtype=torch.uint8),
             cos_sin=torch.zeros(9, 2, 32), positions=None, axis=None, q_norm=None)
    page = 32
    t.update(change)
    return t, page


def calls(bq, t, page):
    tail = (t["starts"], t["lens"], t["table"])
    yield "write", lambda: bq.rope_write_kv_cache(t["q"], t["k"], t["v"], t["out"], t["k_cache"], t["v_cache"], *tail, page,
                                                  cos_sin=t["cos_sin"], positions=t["positions"], axis=t["axis"], q_norm=t["q_norm"])
    yield "read", lambda: bq.read_kv_cache(t["k_cache"], t["v_cache"], t["k"], t["v"], *tail, page)
    yield "decode", lambda: bq.paged_attention_decode(t["q"], t["k_cache"], t["v_cache"], t["out"], *tail, t["workspace"], 2, page)
    yield "prefill", lambda: bq.paged_attention_prefill(t["q"], t["k_cache"], t["v_cache"], t["out"], *tail, 2, page)


@pytest.mark.parametrize("which,error,needle,change", [
    ("write read decode prefill", ValueError, "device", {}),
    ("write read decode prefill", TypeError, "k_cache", dict(k_cache=torch.zeros(8192 * 5, dtype=torch.int8))),
    ("write read decode prefill", ValueError, "v_cache", dict(v_cache=torch.zeros(8192 * 4, dtype=torch.uint8))),
    ("write read decode prefill", ValueError, "whole number", dict(k_cache=torch.zeros(8192 * 5 + 16, dtype=torch.uint8),
                                                                  v_cache=torch.zeros(8192 * 5 + 16, dtype=torch.uint8))),
    ("write read decode prefill", TypeError, "starts", dict(starts=torch.zeros(3, dtype=torch.int64))),
    ("write read decode prefill", ValueError, "lens", dict(lens=torch.zeros(3, dtype=torch.int32))),
    ("write read decode prefill", ValueError, "table", dict(table=torch.zeros(3, 4, dtype=torch.int32))),
    ("write decode prefill", ValueError, "out", dict(out=torch.zeros(3, 4, 48, dtype=torch.bfloat16))),
    ("write decode prefill", TypeError, "q", dict(q=torch.zeros(3, 4, 64))),
    ("write decode prefill", ValueError, "contiguous", dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2))),
    ("write read", ValueError, "v", dict(v=torch.zeros(3, 1, 64, dtype=torch.bfloat16))),
    ("write", ValueError, "cos_sin", dict(cos_sin=torch.zeros(9, 1, 32))),
    ("write", TypeError, "cos_sin", dict(cos_sin=torch.zeros(9, 2, 32, dtype=torch.float64))),
    ("write", ValueError, "positions", dict(positions=torch.zeros(4, dtype=torch.int32))),
    ("write", ValueError, "axis", dict(axis=torch.zeros(32, dtype=torch.uint8))),
    ("write", ValueError, "axis", dict(axis=torch.zeros(31, dtype=torch.uint8), positions=torch.zeros(3, 3, dtype=torch.int32))),
    ("write", ValueError, "q_norm", dict(q_norm=torch.zeros(63, dtype=torch.bfloat16))),
    ("write", ValueError, "q_out", dict(q=None)),
])
def test_binding_refusals(bq, which, error, needle, change):
    t, page = tensors(**change)
    for name, call in calls(bq, t, page):
        if name in which.split():
            with pytest.raises(error, match=needle):
                call()
