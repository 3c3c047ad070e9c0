"""Refusals of the head, cache and attention calls, without a GPU: the binding's checks of metadata (host tensors that pass
them are refused for their placement, before a C call) and the C ABI's checks before it looks for a device."""

import ctypes
import struct

import pytest
import torch

import block_quantized_weight_matmul_amd as q
from block_quantized_weight_matmul_amd import _lib as L
from tests.test_binding_f8 import expect, f32, i32

H = torch.float16


def half(*shape):
    return torch.zeros(shape, dtype=H)


def meta(*shape, dtype=H):
    return torch.empty(shape, dtype=dtype, device="meta")


def cache(pages=4, page=16, heads=2, D=32, dtype=H):
    c = object.__new__(q.KVCache)
    c.pages, c.page, c.heads, c.D, c.dtype, c.device, c._h = pages, page, heads, D, dtype, 0, None
    c._id, c._type = (0, heads, D), 1
    c.k = c.v = c.k_scales = c.v_scales = None
    return c


def test_head_refusals():
    x = f32(3, 4, 32)
    expect(lambda: q.head_norm_rope(x.long(), x, None, None), "q has dtype")
    expect(lambda: q.head_norm_rope(f32(4, 32), x, None, None), "dimensions")
    expect(lambda: q.head_norm_rope([1.0], x, None, None), "torch tensor")
    expect(lambda: q.head_norm_rope(x, x, None, None), "device tensor")


def test_cache_refusals():
    k = half(4, 2, 16, 32)
    expect(lambda: q.KVCache(k.float(), k), "k has dtype")
    expect(lambda: q.KVCache(k, k.bfloat16()), "v has dtype")
    expect(lambda: q.KVCache(k, half(4, 2, 16, 16)), "v has shape")
    expect(lambda: q.KVCache(k[0], k), "dimensions")
    expect(lambda: q.KVCache(k, k, f32(4, 2, 16)), "only an e4m3 cache")
    codes = k.to(torch.uint8)
    expect(lambda: q.KVCache(codes, codes), "torch tensor")
    expect(lambda: q.KVCache(codes, codes, f32(4, 2, 16), f32(4, 2, 8)), "v_scales has shape")
    expect(lambda: q.KVCache(codes, codes, f32(4, 2, 16), half(4, 2, 16)), "v_scales has dtype")
    expect(lambda: q.KVCache(k, k), "device tensor")
    expect(lambda: q.KVCache.empty(4, 16, 2, 32, torch.float32, "cpu"), "cache dtype")
    c = cache()
    expect(lambda: c.write(half(3, 2, 32).long(), half(3, 2, 32), i32(3)), "k has dtype")
    expect(lambda: c.write(half(3, 2, 32), half(3, 2, 32), i32(3)), "device tensor")
    expect(lambda: c.read(i32(2, 4), i32(3).long(), 5), "starts has dtype")
    expect(lambda: c.read(i32(2, 4), i32(0), 5), "starts is empty")
    expect(lambda: c.read(i32(3, 4), i32(3), 5), "table has 3 rows")
    expect(lambda: c.read(i32(2, 4).long(), i32(3), 5), "table has dtype")
    expect(lambda: c.read(i32(2, 4), i32(3), 5), "device tensor")
    expect(lambda: c.attend(f32(2, 4, 32), i32(2, 4), i32(2)), "q has dtype")
    expect(lambda: c.attend(half(2, 4, 32), i32(2, 4), i32(2)), "device tensor")
    expect(lambda: c.norm_rope_write(half(2, 4), half(2, 2, 32), half(2, 2, 32), i32(2), None, None), "dimensions")


def test_prompt_refusals():
    x = half(3, 4, 32)
    expect(lambda: q.attend_prompt(x.float(), x, x, i32(2)), "q has dtype")
    expect(lambda: q.attend_prompt(x[0], x, x, i32(2)), "dimensions")
    expect(lambda: q.attend_prompt(x, x, x, i32(2)), "device tensor")


class Calls:
    """Buffers for calls that are refused before they are read."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(1 << 12)
        self.p = (ctypes.addressof(self.buf) + 255) & ~255


def test_c_cache_create_errors():
    c = Calls()
    h, p = ctypes.c_void_p(), c.p
    create = L.lib.qmm_cache_create
    good = [ctypes.byref(h), p, p, None, None, 1, 4, 16, 2, 32]

    def refused(at, value, status):
        args = list(good)
        args[at] = value
        assert create(*args) == status, (at, value)
        assert h.value is None

    refused(0, None, -1)
    refused(1, None, -1)
    refused(2, None, -1)
    refused(1, p + 8, -4)
    refused(2, p + 4, -4)
    refused(3, p, -1)       # scales of a 16-bit cache
    for t in (0, 4, -1):
        refused(5, t, -2)
    refused(5, 3, -1)       # e4m3 without scales
    for n in (0, -1, 1 << 27):
        refused(6, n, -3)
    for n in (0, 8, 17, 24, 8192, -16):
        refused(7, n, -3)
    for n in (0, 1025):
        refused(8, n, -3)
    for n in (0, 8, 24, 272):
        refused(9, n, -3)
    assert L.lib.qmm_cache_destroy(None) == 0


def refusals(call, layout, good):
    """refused(changes, status): the call with some of the struct's fields changed."""
    def refused(changes, status):
        args = dict(good)
        args.update(changes)
        assert call(struct.pack(layout, *args.values()), None) == status, changes
    return refused


HEADS = ("q k v q_weight k_weight positions inv_freq slots q_out k_out q_token q_head k_token k_head v_token v_head "
         "T Hq H D R xt wt ot interleaved eps").split()
PROMPT = "q k v q_starts k_starts out q_token q_head k_token k_head v_token v_head B Tq Tk Hq H D dt causal scale".split()


def test_c_null_handles():
    c = Calls()
    lib, a = L.lib, ctypes.string_at(c.p, 256)
    assert lib.qmm_cache_write(None, a, None) == -1
    assert lib.qmm_cache_read(None, a, None) == -1
    assert lib.qmm_cache_attend(None, a, None) == -1
    assert lib.qmm_cache_norm_rope_write(None, a, None) == -1
    assert lib.qmm_cache_attend_workspace_bytes(None, 1, 2, 16) == 0
    assert lib.qmm_head_norm_rope(None, None) == -1
    assert lib.qmm_attend_prompt(None, None) == -1


def test_c_head_errors():
    p = Calls().p
    good = dict(zip(HEADS, [p, p, 0, 0, 0, p, p, 0, p, p, 64, 32, 64, 32, 0, 0, 3, 2, 2, 32, 32, 0, 0, 1, 0, 1e-6]))
    refused = refusals(L.lib.qmm_head_norm_rope, "21q4if4x", good)
    for n in ("q", "k", "positions", "inv_freq", "q_out", "k_out"):
        refused({n: 0}, -1)
    for n in ("q", "k", "positions", "inv_freq"):
        refused({n: p + 2}, -4)
    for n in ("q_weight", "k_weight", "q_out", "k_out"):
        refused({n: p + 1}, -4)
    for n in ("q_token", "q_head", "k_token", "k_head"):
        refused({n: -1}, -3)
        refused({n: 1 << 41}, -3)
    for n in ("xt", "wt", "ot"):
        refused({n: 3}, -2)
        refused({n: -1}, -2)
    for n, values in (("T", (-1, 1 << 31)), ("Hq", (-1, 1025)), ("H", (-1, 1025)), ("D", (0, 24, 272)), ("R", (-8, 4, 40))):
        for v in values:
            refused({n: v}, -3)
    for v in (-1.0, float("nan"), float("inf")):
        refused({"eps": v}, -1)
    refused({"interleaved": 2}, -1)
    refused({"Hq": 0, "H": 0}, -3)
    refused({"T": 0, "q": 0, "k": 0, "positions": 0, "inv_freq": 0, "q_out": 0, "k_out": 0}, 0)  # nothing to look at


def test_c_prompt_errors():
    p = Calls().p
    good = dict(zip(PROMPT, [p, p, p, p, p, p, 64, 32, 64, 32, 64, 32, 1, 3, 3, 2, 2, 32, 1, 1, 0.2]))
    refused = refusals(L.lib.qmm_attend_prompt, "18q2if4x", good)
    for n in ("q", "k", "v", "q_starts", "k_starts", "out"):
        refused({n: 0}, -1)
        refused({n: p + 1}, -4)
    for n in ("k", "v"):
        refused({n: p + 8}, -4)
    for n in ("k_token", "k_head", "v_token", "v_head"):
        refused({n: 68}, -4)
    for n in ("k_token", "v_token"):
        refused({n: 16}, -3)
        refused({n: 1 << 24}, -3)
    for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head"):
        refused({n: -8}, -3)
    for t in (0, 3, -1):
        refused({"dt": t}, -2)
    for n, values in (("B", (-1, 1 << 21)), ("Tq", (-1, 1 << 31)), ("Tk", (-1, 1 << 31)), ("Hq", (0, 3, 8193)), ("H", (0, 3, 1025)),
                      ("D", (0, 8, 40, 512))):
        for v in values:
            refused({n: v}, -3)
    refused({"causal": 2}, -1)
    for v in (0.0, -1.0, float("nan"), float("inf")):
        refused({"scale": v}, -1)
    none = {n: 0 for n in PROMPT[:6]}
    refused({"B": 0, **none}, 0)
    refused({"Tq": 0, **none}, 0)


def test_checks_in_order_of_use():
    """Meta tensors pass the checks of type and dimension and stop at the device."""
    with pytest.raises(ValueError, match="device tensor"):
        q.attend_prompt(meta(3, 4, 32), meta(3, 4, 32), meta(3, 4, 32), i32(2))
