"""Refusals of the e4m3 and router calls, without a GPU: the binding's checks of metadata (host tensors that pass them
are refused for their placement, before a C call) and the C ABI's checks before it looks for a device."""

import ctypes
import subprocess
import sys

import pytest
import torch

import block_quantized_weight_matmul_amd as q
from block_quantized_weight_matmul_amd import _lib as L
from tests.conftest import ROOT


def expect(fn, text):
    with pytest.raises(ValueError, match=text):
        fn()


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def matrix(M, K, E=1):
    m = object.__new__(q.F8Matrix)
    m.M, m.K, m.n_experts, m._h, m.device = M, K, E, None, 0
    return m


def plan(N, S, E):
    return q.RoutePlan(i32(64), N, S, E)


def test_quantize_refusals():
    expect(lambda: q.f8_quantize(torch.zeros((2, 3), dtype=torch.float64)), "x has dtype")
    expect(lambda: q.f8_quantize(f32(4)), "dimensions")
    expect(lambda: q.f8_quantize(f32(4, 0)), "no columns")
    expect(lambda: q.f8_quantize(f32(4, 8)), "device tensor")
    expect(lambda: q.f8_quantize([1.0]), "torch tensor")
    expect(lambda: q.F8Matrix.quantize(f32(4, 8)), "device tensor")
    expect(lambda: q.F8Matrix.quantize(f32(4)), "dimensions")
    p = plan(4, 2, 3)
    expect(lambda: q.f8_quantize_t(f32(5, 8), p), "5 rows")
    expect(lambda: q.f8_quantize_t(f32(4, 3, 8), p), "x has shape")
    expect(lambda: q.f8_quantize_t(f32(4, 8), p), "device tensor")


def test_matrix_refusals():
    codes, scales = torch.zeros((130, 256), dtype=torch.uint8), f32(2, 2)
    expect(lambda: q.F8Matrix(codes.float(), scales, 130, 200), "codes has dtype")
    expect(lambda: q.F8Matrix(codes, scales, 130, 100), "codes has shape")
    expect(lambda: q.F8Matrix(codes, f32(1, 2), 130, 200), "scales has shape")
    expect(lambda: q.F8Matrix(codes, scales.half(), 130, 200), "scales has dtype")
    expect(lambda: q.F8Matrix(codes, scales, 130, 200, 2), "3 dimensions")
    expect(lambda: q.F8Matrix(codes, scales, 0, 200), "positive")
    expect(lambda: q.F8Matrix(codes, scales, 130, 200), "device tensor")


def test_product_refusals():
    m = matrix(48, 200)
    expect(lambda: m.linear(f32(3, 201)), "matrix has K")
    expect(lambda: m.linear(f32(200)), "dimensions")
    expect(lambda: m.linear(torch.zeros((3, 200), dtype=torch.int8)), "x has dtype")
    expect(lambda: m.linear(f32(3, 200)), "device tensor")
    expect(lambda: m.gemm(f32(3, 200)), "f8_quantize")
    st = matrix(48, 200, 4)
    expect(lambda: st.linear(f32(3, 200)), "stacks 4")
    expect(lambda: st.linear_id(f32(3, 200), i32(3, 2).long()), "ids has dtype")
    expect(lambda: st.linear_id(f32(4, 200), i32(3, 2)), "x has shape")
    expect(lambda: st.linear_id(f32(3, 3, 200), i32(3, 2)), "x has shape")
    expect(lambda: st.linear_id(f32(3, 200), i32(3, 0)), "no slots")
    expect(lambda: st.linear_id(f32(3, 200), i32(3, 2)), "device tensor")
    t = object.__new__(q.F8Tokens)
    t.ptrs, t.pitch, t.rows, t.length, t.plan, t.device = (0, 0), 256, 3, 200, None, 0
    expect(lambda: st.gemm_id(t, plan(3, 2, 5)), "plan has 5 experts")
    expect(lambda: st.gemm_id(t, plan(4, 2, 4)), "3 rows")
    expect(lambda: matrix(48, 199).gemm(t), "tokens have K=200")
    expect(lambda: m.update(f32(48, 201)), "w has shape")
    expect(lambda: q.f8_wgrad(t, t, plan(3, 2, 5)), "quantized with the plan")


def test_route_refusals():
    expect(lambda: q.route(f32(4), 1), "dimensions")
    expect(lambda: q.route(f32(4, 8), 2), "device tensor")
    expect(lambda: q.route(f32(4, 8).long(), 2), "dtype")
    expect(lambda: q.route_plan(i32(4, 2).long(), 8), "dtype")
    expect(lambda: q.route_plan(i32(4, 2), 8), "device tensor")
    expect(lambda: q.route_plan(i32(4, 0), 8), "a slot")
    expect(lambda: q.balance_loss(i32(8), f32(8), 2, 0.1), "counts has shape")
    expect(lambda: q.route_combine(f32(4, 8)), "dimensions")
    expect(lambda: q.route_combine(f32(4, 2, 8), f32(4, 2)), "device tensor")
    expect(lambda: q.route_combine_backward(f32(4, 2, 8), None, f32(4, 8)), "weights are needed")


def test_c_argument_errors():
    lib = L.lib
    buf = ctypes.create_string_buffer(1 << 12)
    p = (ctypes.addressof(buf) + 255) & ~255
    h = ctypes.c_void_p()
    assert lib.qmm_f8_padded(0) == 0 and lib.qmm_f8_padded(-5) == 0
    assert [lib.qmm_f8_padded(n) for n in (1, 128, 129)] == [128, 128, 256]
    assert lib.qmm_f8_create(None, p, p, 1, 4, 4) == -1
    assert lib.qmm_f8_create(ctypes.byref(h), None, p, 1, 4, 4) == -1
    assert lib.qmm_f8_create(ctypes.byref(h), p + 8, p, 1, 4, 4) == -4
    assert lib.qmm_f8_create(ctypes.byref(h), p, p, 0, 4, 4) == -3
    assert lib.qmm_f8_create(ctypes.byref(h), p, p, 1, 0, 4) == -3
    assert lib.qmm_f8_create(ctypes.byref(h), p, p, 1, 4, 1 << 22) == -3
    assert lib.qmm_f8_destroy(None) == 0
    assert lib.qmm_f8_quantize(p, 3, 8, 2, 8, p, p, None, None, None) == -2
    assert lib.qmm_f8_quantize(p, 0, 7, 2, 8, p, p, None, None, None) == -3      # rows overlap
    assert lib.qmm_f8_quantize(p, 0, 8, 2, 0, p, p, None, None, None) == -3
    assert lib.qmm_f8_quantize(p, 0, 8, -1, 8, p, p, None, None, None) == -3
    assert lib.qmm_f8_quantize(p, 0, 8, 2, 8, p, None, None, None, None) == -1   # codes without scales
    assert lib.qmm_f8_quantize(p, 0, 8, 2, 8, None, None, None, None, None) == -1
    assert lib.qmm_f8_quantize(p + 2, 0, 8, 2, 8, p, p, None, None, None) == -4
    assert lib.qmm_f8_quantize(p, 0, 8, 2, 8, p + 8, p, None, None, None) == -4
    assert lib.qmm_f8_quantize(None, 0, 8, 0, 8, None, None, None, None, None) == 0  # nothing to do
    assert lib.qmm_f8_quantize_weight(p, 0, 1, 4, 4, None, None, None, None, None) == -1
    for fn, args in ((lib.qmm_f8_gemm, (None, p, p, 1, p, 0, None, 0, None)),
                     (lib.qmm_f8_linear, (None, p, 0, 8, 1, p, 0, None, 0, None)),
                     (lib.qmm_f8_gemm_id, (None, p, p, 1, 1, 1, p, p, 0, None)),
                     (lib.qmm_f8_linear_id, (None, p, 0, 1, 1, 1, p, p, 0, None, 0, None)),
                     (lib.qmm_f8_transpose, (None, p, p, None)), (lib.qmm_f8_dequantize, (None, 0, p, 0, None))):
        assert fn(*args) == -1 and b"handle" in lib.qmm_last_error()
    assert lib.qmm_f8_linear_workspace_bytes(None, 4) == 0
    assert lib.qmm_route_plan_bytes(8, 1025) == 0 and lib.qmm_route_plan_bytes(-1, 4) == 0
    need = lib.qmm_route_plan_bytes(8, 4)
    assert need > 0
    assert lib.qmm_route_plan(p, 4, 2, 4, p, need - 4, None) == -1
    assert lib.qmm_route_plan(p, 4, 65, 4, p, 1 << 20, None) == -3
    assert lib.qmm_route_plan(p, 4, 2, 1025, p, 1 << 20, None) == -3
    assert lib.qmm_route_plan(p, 1 << 22, 2, 4, p, 1 << 40, None) == -3
    assert lib.qmm_f8_wgrad(p, p, p, p, 1 << 24, 4, 4, p, 0, None, 0, None) == -3
    assert lib.qmm_f8_wgrad(p, p, p, p, 4, 4, 4, p, 5, None, 0, None) == -2
    assert lib.qmm_f8_wgrad(p, p, None, p, 4, 4, 4, p, 0, None, 0, None) == -1
    need = lib.qmm_f8_wgrad_workspace_bytes(1 << 14, 128, 256)
    assert need > 0 and lib.qmm_f8_wgrad_workspace_bytes(0, 128, 256) == 0
    assert lib.qmm_f8_wgrad(p, p, p, p, 1 << 14, 128, 256, p, 0, p, need - 4, None) == -1
    assert lib.qmm_f8_wgrad(p, p, p, p, 1 << 14, 128, 256, p, 0, p + 4, need, None) == -4
    assert lib.qmm_f8_wgrad_id(p, p, p, p, 4, 1, 4, 4, 4, None, p, 0, None) == -1
    assert lib.qmm_route(p, 0, 4, 8, 9, None, 1, 0.0, p, p, p, p, p, p, 1 << 20, None) == -3   # S > E
    assert lib.qmm_route(p, 0, 4, 128, 65, None, 1, 0.0, p, p, p, p, p, p, 1 << 20, None) == -3
    assert lib.qmm_route(p, 0, 4, 8, 2, None, 2, 0.0, p, p, p, p, p, p, 1 << 20, None) == -1
    assert lib.qmm_route(p, 0, 4096, 8, 2, None, 1, 0.0, p, p, p, p, p, p, 0, None) == -1      # workspace
    assert lib.qmm_route(p, 0, 4096, 8, 2, None, 1, 0.0, p, p, p, p, p, p + 4, 1 << 20, None) == -4
    assert lib.qmm_route_combine(p, 2, p, 1, 4, 2, 8, p, None) == -2                            # weights' type
    assert lib.qmm_route_combine(p, 0, None, 0, 4, 0, 8, p, None) == -3
    assert lib.qmm_route_combine_backward(p, 0, None, 0, 4, 2, 8, p, p, p, None) == -1
    # a call takes no bf16 that took none before
    assert lib.qmm_gemv(None, p, 2, 1, p, None) == -1


def test_row_layouts_need_no_device():
    x = f32(4, 8)
    from block_quantized_weight_matmul_amd import f8
    expect(lambda: f8._rows(x, "x"), "device tensor")


def test_route_backward_refuses_other_types():
    """The kernels read counts and ids as int32: a sum over stacked counts is int64."""
    l, ids, w, counts = f32(4, 8), i32(4, 2), f32(4, 2), i32(9)
    r = q.Routing(ids, w, counts, f32(8), f32(), True, 0.1, None)
    summed = torch.stack([counts, counts]).sum(0)
    assert summed.dtype == torch.int64
    expect(lambda: q.route_backward(l, r._replace(counts=summed), w, f32(1)), "counts has dtype")
    expect(lambda: q.route_backward(l, r._replace(counts=counts.float()), w, f32(1)), "counts has dtype")
    expect(lambda: q.route_backward(l, r._replace(ids=ids.long()), w, f32(1)), "ids has dtype")
    expect(lambda: q.route_backward(l, r._replace(ids=i32(8)), w, f32(1)), "ids must be a tensor of 2")
    expect(lambda: q.route_backward(l, r._replace(valid=i32(4)), w, f32(1)), "valid has dtype")


def test_quantized_operands_of_a_plan_have_its_sizes():
    """The products take the width of a row of codes from the plan's sizes: operands of another width would be read at
    wrong places and past their end."""
    p = plan(40, 2, 3)
    assert p.routed == 128 * 5 and p.routed % 128 == 0
    u8 = torch.uint8

    def tokens(width, length):
        return lambda: q.F8Tokens(torch.zeros((6, width), dtype=u8), f32(width // 128, 6), 6, length, p)

    expect(tokens(128, 80), "codes has shape")               # the pairs padded to 128, not the experts' own
    expect(tokens(p.routed + 128, 80), "codes has shape")
    expect(tokens(p.routed, 79), "79 tokens")
    expect(tokens(p.routed, 40), "40 tokens")
    expect(tokens(p.routed, 80), "device tensor")            # right: only its place is not


def test_plan_refuses_other_buffers():
    """The products read tile lists and pairs from a plan: its buffer has qmm_route_plan_bytes, as int32."""
    need = L.lib.qmm_route_plan_bytes(80, 3) // 4
    expect(lambda: q.RoutePlan(i32(need).long(), 40, 2, 3), "data has dtype")
    expect(lambda: q.RoutePlan(i32(need, 1), 40, 2, 3), "dimensions")
    expect(lambda: q.RoutePlan([0] * need, 40, 2, 3), "torch tensor")
    expect(lambda: q.RoutePlan(i32(need - 4), 40, 2, 3).place(0), "need")
    expect(lambda: q.RoutePlan(i32(need), 60, 2, 3).place(0), "need")
    expect(lambda: q.RoutePlan(i32(need), 40, 2, 1025).place(0), "need")       # no such plan
    expect(lambda: q.RoutePlan(i32(need), 40, 2, 3).place(0), "device tensor")  # right: only its place is not
    # and the calls that read one ask for it
    short, m = q.RoutePlan(i32(need - 4), 40, 2, 3), matrix(6, 200, 3)
    t = object.__new__(q.F8Tokens)
    t.ptrs, t.pitch, t.rows, t.length, t.plan, t.device, t.transposed = (0, 0), 256, 40, 200, None, 0, None
    expect(lambda: m.gemm_id(t, short), "need")
    t = object.__new__(q.F8Tokens)
    t.ptrs, t.pitch, t.rows, t.length, t.plan, t.device, t.transposed = (0, 0), short.routed, 6, 80, short, 0, None
    expect(lambda: q.f8_wgrad(t, t, short), "need")


def test_transpose_refuses_shared_buffers():
    """Codes and scales are read while the transpose's are written: none of the four buffers may share memory."""
    from block_quantized_weight_matmul_amd import f8

    def square(codes, scales):
        m = matrix(256, 256)
        m.codes, m.scales, m._spans = codes, scales, f8._spans(codes, scales)
        return m

    u8 = torch.uint8
    room, other = torch.zeros((512, 256), dtype=u8), torch.zeros((256, 256), dtype=u8)
    m = square(room[:256], f32(2, 2))
    expect(lambda: m.transposed(m), "buffers of its own")
    expect(lambda: m.transposed(square(m.codes, f32(2, 2))), "buffers of its own")
    expect(lambda: m.transposed(square(room[128:384], f32(2, 2))), "buffers of its own")
    expect(lambda: m.transposed(square(other, m.scales)), "buffers of its own")
    expect(lambda: m.transposed(square(other, room[:1, :16].view(torch.float32).view(2, 2))), "buffers of its own")
    other_device = square(room[256:], f32(2, 2))
    m._check_transpose(other_device)             # buffers of its own
    other_device.device = 1
    expect(lambda: m.transposed(other_device), "on cuda:1")


def test_operands_quantized_along_the_other_axis():
    """Where N equals K (or M) the shapes do not tell f8_quantize from f8_quantize_t: what made them does."""
    def square(transposed):
        t = object.__new__(q.F8Tokens)
        t.ptrs, t.pitch, t.rows, t.length, t.plan, t.device, t.transposed = (0, 0), 256, 200, 200, None, 0, transposed
        return t

    along_k, along_tokens, own = square(False), square(True), square(None)
    expect(lambda: matrix(48, 200).gemm(along_tokens), "along K")
    expect(lambda: matrix(48, 200, 4).gemm_id(along_tokens, plan(200, 1, 4)), "along K")
    expect(lambda: q.f8_wgrad(along_k, along_tokens), "along the tokens")
    expect(lambda: q.f8_wgrad(along_tokens, along_k), "along the tokens")
    for t in (along_k, own):     # accepted: refused for the plan's buffer only
        expect(lambda: matrix(48, 200, 4).gemm_id(t, plan(200, 1, 4)), "need")


def test_import_needs_no_private_names_of_torch():
    """Without torch's private shortcuts for the current device and stream the binding takes the public calls."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import block_quantized_weight_matmul_amd as q
from block_quantized_weight_matmul_amd import f8

class Stream:
    cuda_stream = 77

torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device: Stream if device == 3 else None
seen = []
f8._call(3, lambda *a: seen.append(a) or 0, 1, 2)
assert seen == [(1, 2, 77)], seen
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_sizes_kept_between_calls_are_bounded():
    """A server with any number of tokens meets ever new sizes: what is kept of them does not grow with it."""
    from block_quantized_weight_matmul_amd import f8, routing
    for n in range(1, 3000):
        q.RoutePlan(i32(4), n, 1, 5)
    assert len(routing._plan_sizes) <= 1024
    assert q.RoutePlan(i32(4), 7, 1, 5).bytes == L.lib.qmm_route_plan_bytes(7, 5)
    assert all(type(d) is f8._Seen for d in (routing._plan_sizes, routing._route_need, f8._wgrad_need))
    d = f8._Seen()
    for n in range(3000):
        v = d[n] = n + 1
        assert v == n + 1 and d.get(n) == n + 1 and len(d) <= 1024


def test_plan_holds_what_is_read():
    """Counts, offsets, first tiles, the pairs in order, lists of the tiles of 32, 64 and 128 pairs, and above 32768 pairs
    the counts of the chunks that its three launches share."""
    for pairs, E in ((1, 1), (80, 3), (16384, 128), (32768, 8), (32769, 8), (1 << 22, 1024)):
        B = E + 2
        words = B + 2 * (B + 1) + 3 + pairs + sum(3 * (pairs // t + min(B, pairs)) for t in (32, 64, 128))
        if pairs > 32768:
            per = -(-pairs // 256)
            words += -(-pairs // (-(-per // 1024) * 1024)) * B
        assert L.lib.qmm_route_plan_bytes(pairs, E) == -(-words // 4) * 16, (pairs, E)


def test_a_shared_handle_is_not_freed_twice(monkeypatch):
    seen = []
    monkeypatch.setattr(L.lib, "qmm_f8_destroy", lambda h: seen.append(h.value) or 0)
    m = matrix(48, 200)
    m._h = ctypes.c_void_p(4096)
    twin = object.__new__(q.F8Matrix)
    twin.__dict__.update(m.__dict__)
    m.close()
    twin.close()
    m.close()
    assert seen == [4096]
    assert twin.handle is None or twin.handle.value is None     # refused by the library: no handle
