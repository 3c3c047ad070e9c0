"""e4m3 operands with a scale per block of 128 on the device: quantizers bit for bit, products and gradients against
the fp64 oracle within the bound its arithmetic allows (oracle.f8.product_bound, plus half a step of the output's type)."""

import numpy as np
import pytest
import torch

import block_quantized_weight_matmul_amd as q
from oracle import f8 as O
from tests.gpu_helpers import to_host

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def host64(t):
    return to_host(t.double())


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def check(y, ref, bound, label=""):
    """bound: an array, or a pair: for 32-bit outputs and for 16-bit ones (which the 8-bit matrix cores compute)."""
    if isinstance(bound, tuple):
        bound = bound[y.dtype != torch.float32]
    got = host64(y)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    tol = bound + (np.abs(ref) + bound) * HALF_STEP[y.dtype] + SMALLEST[y.dtype]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{label}: {bad.sum()} of {got.size}; worst {np.nanmax(np.abs(got - ref) / tol)} of the bound"


def bounds(xv, wv):
    return O.product_bound(xv, wv), O.product_bound(xv, wv, f8_cores=True)


def same(codes, scales, want, label=""):
    wc, ws = want
    gc, gs = to_host(codes), to_host(scales)
    assert gs.shape == ws.shape and gc.shape == wc.shape, label
    assert np.array_equal(gs.view(np.uint32)[~np.isnan(ws)], ws.view(np.uint32)[~np.isnan(ws)]), f"{label}: scales"
    assert np.array_equal(np.isnan(gs), np.isnan(ws)), f"{label}: NaN scales"
    if np.isnan(ws).any():   # a block that holds an Inf or a NaN: its codes are not specified
        keep = np.repeat(~np.isnan(ws.T), 128, 1)   # token scales: [groups, rows]
        gc, wc = gc[keep], wc[keep]
    assert np.array_equal(gc, wc), f"{label}: {(gc != wc).sum()} codes differ"


def tricky(g, N, K):
    """Normal values with ties (multiples of 1/64 of the largest), zeros, tiny and large rows."""
    x = g.standard_normal((N, K))
    x[::3] = np.round(x[::3] * 64) / 64
    x[1::5] *= 2.0 ** -12
    x[2::7] = 0.0
    x[:, ::41] *= 16.0
    return x


SHAPES = [(1, 1), (1, 128), (3, 127), (5, 129), (16, 256), (33, 515), (129, 130), (300, 1111), (128, 2560)]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,K", SHAPES)
def test_quantize_bits(N, K, dtype):
    g = np.random.default_rng([11, N, K])
    x = dev(tricky(g, N, K), DTYPES[dtype])
    xv = host64(x)
    rows, cols = q.f8_quantize_pair(x)
    same(rows.codes, rows.scales, O.quantize_rows(xv), "rows")
    same(cols.codes, cols.scales, O.quantize_rows(xv.T), "columns")
    only = q.f8_quantize(x)
    assert torch.equal(only.codes, rows.codes) and torch.equal(only.scales, rows.scales)
    only = q.f8_quantize_t(x)
    assert torch.equal(only.codes, cols.codes) and torch.equal(only.scales, cols.scales)
    want = O.rows_values(*O.quantize_rows(xv), K)
    assert np.all(np.abs(host64(rows.values()) - want) <= np.abs(want) * 2.0 ** -24)


def test_quantize_every_quotient():
    """Ties and their fp32 neighbours: values m * s for every middle m of two codes, and the floats around them."""
    v = O.e4m3_values()[:127]
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    for amax in (448.0, 1.0, 3.0e-7, 1.7e30, 0.7315):
        s = np.float32(O.scale(np.array([amax]))[0])
        m = (mid.astype(np.float64) * s).astype(np.float32)
        x = np.stack([m, np.nextafter(m, np.float32(np.inf)), np.nextafter(m, np.float32(0)), -m]).T
        x = np.concatenate([np.full((126, 1), amax, np.float32), x], 1)
        t = q.f8_quantize(dev(x))
        same(t.codes, t.scales, O.quantize_rows(x), f"amax {amax}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_16_bit_quotient(dtype):
    """Every value of the 17 octaves below the block's largest, which takes every significand (bf16) or every 16th (fp16):
    448 x / amax is a middle of two codes often, down to the smallest codes."""
    bits, step = (7, 1) if dtype == "bf16" else (10, 16)
    largest = 1.0 + np.arange(0, 2 ** bits, step) / 2.0 ** bits
    x = np.outer(2.0 ** -np.arange(0.0, 17.0), 1.0 + np.arange(2 ** bits) / 2.0 ** bits).ravel()
    rows = []
    for i, a in enumerate(largest):
        v = x[x <= a]
        v = np.concatenate([v, np.zeros(-v.size % 127)]).reshape(-1, 127) * np.where(i % 2, -1.0, 1.0)
        rows.append(np.concatenate([np.full((len(v), 1), a), v], 1))
    t = dev(np.concatenate(rows), DTYPES[dtype])
    same(*(lambda c: (c.codes, c.scales))(q.f8_quantize(t)), O.quantize_rows(host64(t)))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_quantize_extremes(dtype):
    big = {"f32": 3.0e38, "f16": 65504.0, "bf16": 3.0e38}[dtype]
    x = np.zeros((6, 400))
    x[0, 0], x[0, 1], x[0, 2] = big, -big / 2, big / 3
    x[1, 200], x[1, 201] = 1e-30, -3e-31
    x[2, 5] = np.inf
    x[3, 130] = np.nan
    x[4, 399] = -np.inf
    x[5] = 2.0 ** -24
    t = dev(x, DTYPES[dtype])
    rows, cols = q.f8_quantize_pair(t)
    same(rows.codes, rows.scales, O.quantize_rows(host64(t)))
    same(cols.codes, cols.scales, O.quantize_rows(host64(t).T))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_quantize_strided_rows(dtype):
    g = np.random.default_rng(12)
    wide = dev(tricky(g, 37, 700), DTYPES[dtype])
    for lo, hi in ((0, 700), (8, 400), (1, 300), (699, 700)):
        x = wide[:, lo:hi]
        rows, cols = q.f8_quantize_pair(x)
        same(rows.codes, rows.scales, O.quantize_rows(host64(x)), (lo, hi))
        same(cols.codes, cols.scales, O.quantize_rows(host64(x).T), (lo, hi))
    x = wide[::2]
    assert torch.equal(q.f8_quantize(x).codes, q.f8_quantize(x.contiguous()).codes)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("E,M,K", [(1, 1, 1), (1, 128, 128), (1, 130, 257), (3, 200, 515), (2, 127, 1024)])
def test_weight_bits(E, M, K, dtype):
    g = np.random.default_rng([13, E, M, K])
    w = dev(g.standard_normal((E, M, K)) * 0.02, DTYPES[dtype])
    m = q.F8Matrix.quantize(w)
    wv = host64(w)
    t = m.transposed()
    u = q.F8Matrix(torch.full_like(t.codes, 99), torch.zeros_like(t.scales), K, M, E)
    m.update(w, transposed=u)
    for e in range(E):
        same(m.codes[e], m.scales[e], O.quantize_weight(wv[e]), "weights")
        want = O.quantize_weight(wv[e].T)
        same(t.codes[e], t.scales[e], want, "transpose")
        same(u.codes[e], u.scales[e], want, "transpose of update")
        value = O.weight_values(*O.quantize_weight(wv[e]), K)
        for dt in DTYPES.values():
            check(m.dequantize(e, dt), value, np.abs(value) * 2.0 ** -24, "dequantize")


def weights(g, M, K):
    w = g.standard_normal((M, K)) * 0.02
    codes, scales = O.quantize_weight(w)
    return q.F8Matrix(dev_u8(codes), dev(scales), M, K), O.weight_values(codes, scales, K)


def dev_u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


TOKENS = [1, 2, 5, 8, 16, 17, 32, 33, 64, 100, 129, 256, 300]


@pytest.mark.parametrize("N", TOKENS)
@pytest.mark.parametrize("M,K", [(64, 128), (1000, 1111), (130, 515), (257, 2560), (1, 1), (4, 40)])
def test_linear_and_gemm(N, M, K):
    g = np.random.default_rng([14, N, M, K])
    m, wv = weights(g, M, K)
    for i, dt in enumerate(DTYPES.values()):
        x = dev(g.standard_normal((N, K)), dt)
        xv = O.rows_values(*O.quantize_rows(host64(x)), K)
        ref, bound = xv @ wv.T, bounds(xv, wv)
        y = torch.full((N, M), float("nan"), dtype=dt, device="cuda")
        m.linear(x, out=y)
        check(y, ref, bound, f"linear {dt}")
        assert torch.equal(y, m.linear(x)), "two calls, two results"
        out = list(DTYPES.values())[(i + 1) % 3]
        check(m.gemm(q.f8_quantize(x), out_dtype=out), ref, bound, f"gemm to {out}")


@pytest.mark.parametrize("N,M,K", [(1, 2560, 9728), (3, 1024, 8192), (16, 2560, 9728), (48, 512, 9728), (200, 512, 9728)])
def test_linear_long_rows(N, M, K):
    g = np.random.default_rng([15, N])
    m, wv = weights(g, M, K)
    x = dev(g.standard_normal((N, K)), torch.float16)
    xv = O.rows_values(*O.quantize_rows(host64(x)), K)
    check(m.linear(x, out_dtype=torch.float32), xv @ wv.T, bounds(xv, wv))


def test_linear_strided_and_unaligned():
    g = np.random.default_rng(16)
    M, K = 96, 300
    m, wv = weights(g, M, K)
    wide = dev(g.standard_normal((40, 3 * K)), torch.bfloat16)
    for n, lo in ((1, 5), (4, 8), (40, K), (40, 2 * K)):
        x = wide[:n, lo:lo + K]
        xv = O.rows_values(*O.quantize_rows(host64(x)), K)
        y = torch.zeros(n * M + 1, dtype=torch.bfloat16, device="cuda")[1:].view(n, M)  # 2-byte aligned output
        m.linear(x, out=y)
        check(y, xv @ wv.T, bounds(xv, wv), (n, lo))


def test_rows_behind_the_last_token_stay():
    g = np.random.default_rng(17)
    m, _ = weights(g, 100, 256)
    for n in (1, 7, 20, 130):
        y = torch.full((n + 3, 100), 7.0, device="cuda")
        m.linear(dev(g.standard_normal((n, 256))), out=y[:n])
        assert bool((y[n:] == 7.0).all()) and not bool((y[:n] == 7.0).any())


def test_bad_token_poisons_its_row_only():
    g = np.random.default_rng(18)
    m, _ = weights(g, 70, 300)
    for n in (3, 40, 200):
        x = g.standard_normal((n, 300))
        x[1, 17], x[2, 299] = np.nan, np.inf
        y = to_host(m.linear(dev(x)))
        assert np.isnan(y[1:3]).all() and np.isfinite(np.delete(y, (1, 2), 0)).all()


def test_no_tokens():
    g = np.random.default_rng(19)
    m, _ = weights(g, 10, 20)
    assert m.linear(torch.empty((0, 20), device="cuda")).shape == (0, 10)
    t, tt = q.f8_quantize_pair(torch.empty((0, 20), device="cuda"))
    assert m.gemm(t).shape == (0, 10)
    dw = q.f8_wgrad(q.f8_quantize_t(torch.empty((0, 10), device="cuda")), tt, out=torch.full((10, 20), 5.0, device="cuda"))
    assert bool((dw == 0).all())


# ---- experts -----------------------------------------------------------------------------------

def stack(g, E, M, K):
    codes, scales, values = [], [], []
    for _ in range(E):
        c, s = O.quantize_weight(g.standard_normal((M, K)) * 0.02)
        codes.append(c)
        scales.append(s)
        values.append(O.weight_values(c, s, K))
    return q.F8Matrix(dev_u8(np.stack(codes)), dev(np.stack(scales)), M, K, E), values


def id_reference(xv, ids, values, M):
    N, S = ids.shape
    ref, bound, coarse = (np.zeros((N, S, M)) for _ in range(3))
    for e, w in enumerate(values):
        t, s = np.nonzero(ids == e)
        if len(t):
            rows = xv[t, s] if xv.ndim == 3 else xv[t]
            ref[t, s] = rows @ w.T
            bound[t, s], coarse[t, s] = bounds(rows, w)
    return ref, (bound, coarse)


def quantized_values(x):
    flat = host64(x).reshape(-1, x.shape[-1])
    return O.rows_values(*O.quantize_rows(flat), x.shape[-1]).reshape(tuple(x.shape))


ID_CASES = [  # N, S, E, M, K
    (1, 1, 1, 16, 32), (1, 8, 128, 64, 512), (4, 8, 32, 300, 512), (5, 3, 4, 130, 200), (40, 2, 3, 70, 1111),
    (16, 8, 8, 100, 256), (64, 4, 16, 129, 384), (300, 2, 5, 64, 130), (700, 1, 2, 20, 40), (2, 64, 100, 32, 128)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("N,S,E,M,K", ID_CASES)
def test_expert_products(N, S, E, M, K, per_slot):
    g = np.random.default_rng([20, N, S, E])
    m, values = stack(g, E, M, K)
    ids = g.integers(0, E, (N, S)).astype(np.int32)   # duplicates among a token's slots too
    if N > 1:
        ids[g.random((N, S)) < 0.15] = -1
        ids[N // 2, 0] = E           # names no expert
        ids[N // 2 + 1:][:1] = -1    # a padded token
    for dt in DTYPES.values():
        x = dev(g.standard_normal((N, S, K) if per_slot else (N, K)), dt)
        ref, bound = id_reference(quantized_values(x), ids, values, M)
        plan = q.route_plan(dev_u8(ids), E)
        want = np.array([(ids == e).sum() for e in range(E)])
        assert np.array_equal(to_host(plan.counts), want)
        rows = x.reshape(-1, K)
        for y in (m.linear_id(x, dev_u8(ids)), m.gemm_id(q.f8_quantize(rows), plan, out_dtype=dt)):
            none = ids >= E
            assert bool(torch.isnan(y[torch.from_numpy(none).cuda()]).all())
            y = torch.where(torch.from_numpy(none).cuda()[:, :, None], torch.zeros_like(y), y)
            check(y, ref, bound, f"{dt}")


def test_all_slots_empty_or_one_expert():
    g = np.random.default_rng(21)
    E, M, K = 4, 50, 130
    m, values = stack(g, E, M, K)
    for N in (2, 200):
        x = dev(g.standard_normal((N, K)))
        y = m.linear_id(x, torch.full((N, 2), -1, dtype=torch.int32, device="cuda"))
        assert bool((y == 0).all())
        ids = np.full((N, 2), 3, np.int32)
        ref, bound = id_reference(quantized_values(x), ids, values, M)
        check(m.linear_id(x, dev_u8(ids)), ref, bound)


@pytest.mark.parametrize("pairs_per_token", [1, 3])
def test_many_pairs(pairs_per_token):
    """More pairs than one sweep of the plan's workgroups holds: every pair finds its own row."""
    N, S, E, M, K = 110000, pairs_per_token, 5, 4, 8
    g = np.random.default_rng(22)
    m, values = stack(g, E, M, K)
    ids = g.integers(-1, E, (N, S)).astype(np.int32)
    x = dev(g.standard_normal((N, K)))
    ref, bound = id_reference(quantized_values(x), ids, values, M)
    check(m.linear_id(x, dev_u8(ids)), ref, bound)


@pytest.mark.parametrize("E", [1, 130, 1024])
@pytest.mark.parametrize("N,S", [(1024, 1), (1025, 1), (683, 6), (4096, 8), (32769, 1)])
def test_plan_sizes(N, S, E):
    """Around the numbers of pairs at which the plan takes another workgroup, and another way."""
    g = np.random.default_rng([23, N, E])
    M, K = 8, 16
    m, values = stack(g, E, M, K)
    ids = g.integers(-1, E + 1, (N, S)).astype(np.int32)
    plan = q.route_plan(dev_u8(ids), E)
    assert np.array_equal(to_host(plan.counts), np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E))
    assert torch.equal(plan.data[:E + 2], q.route_plan(dev_u8(ids), E).data[:E + 2])
    x = dev(g.standard_normal((N, K)))
    y = m.gemm_id(q.f8_quantize(x), plan)
    none = torch.from_numpy(ids >= E).cuda()
    assert bool(torch.isnan(y[none]).all())
    ref, bound = id_reference(quantized_values(x), ids, values, M)
    check(torch.where(none[:, :, None], torch.zeros_like(y), y), ref, bound)


def test_operands_of_other_tensors():
    """Codes and scales that the caller made: uint8 or float8_e4m3fn, a matrix alone or a stack of one."""
    g = np.random.default_rng(24)
    m, _ = weights(g, 140, 260)
    x = dev(g.standard_normal((50, 260)), torch.float16)
    t = q.f8_quantize(x)
    own = q.F8Tokens(t.codes.clone().view(torch.float8_e4m3fn), t.scales.clone(), 50, 260)
    y = m.gemm(t)
    f8 = q.F8Matrix(m.codes.view(torch.float8_e4m3fn), m.scales, 140, 260)
    one = q.F8Matrix(m.codes[None], m.scales[None], 140, 260, 1)
    assert all(torch.equal(y, a.gemm(b)) for a in (m, f8, one) for b in (t, own))
    ids = torch.zeros((50, 1), dtype=torch.int32, device="cuda")
    assert torch.equal(f8.gemm_id(own, q.route_plan(ids, 1))[:, 0], m.gemm_id(t, q.route_plan(ids, 1))[:, 0])
    assert torch.equal(f8.transposed().codes, m.transposed().codes) and torch.equal(f8.dequantize(), m.dequantize())


# ---- gradients ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,M,K", [(1, 1, 1), (5, 40, 30), (128, 128, 256), (333, 130, 257), (1000, 64, 300)])
def test_gradients(N, M, K, dtype):
    g = np.random.default_rng([23, N, M])
    dt = DTYPES[dtype]
    m, wv = weights(g, M, K)
    x, dy = dev(g.standard_normal((N, K)), dt), dev(g.standard_normal((N, M)) * 0.01, dt)
    xq, xt = q.f8_quantize_pair(x)
    gq, gt = q.f8_quantize_pair(dy)
    gv = O.rows_values(*O.quantize_rows(host64(dy)), M)
    check(m.transposed().gemm(gq, out_dtype=dt), gv @ wv, bounds(gv, wv.T), "dx")
    gtv, xtv = (O.rows_values(*O.quantize_rows(host64(t).T), N) for t in (dy, x))
    for out in DTYPES.values():
        check(q.f8_wgrad(gt, xt, dtype=out), gtv @ xtv.T, bounds(gtv, xtv), f"dw {out}")
    # against the difference of the loss <dy, x W^T> along a direction: linear, so it is exact but for the quantization
    # (half a step of e4m3 on each operand: 2^-4 relative, or 2^-10 of the block's largest / 448)
    v = g.standard_normal((M, K))
    dw = host64(q.f8_wgrad(gt, xt))
    a, b = np.abs(host64(dy)), np.abs(host64(x))
    da, db = a * 2.0 ** -4 + a.max() * 2.0 ** -18, b * 2.0 ** -4 + b.max() * 2.0 ** -18
    slack = (da.T @ b + a.T @ db + da.T @ db) * (1 + 1e-3)
    difference = (host64(dy) * (host64(x) @ v.T)).sum()
    assert abs((dw * v).sum() - difference) <= (slack * np.abs(v)).sum()


def test_gradients_against_differences():
    """Operands of powers of two within a factor of 8 are their codes, so <dy, x W^T> is linear in x and in W as it is
    computed: its differences are the gradients' products with the steps.  Error: a scale's rounding in each of two factors
    of a product (2^-23), up to K or N terms of a sum in fp32."""
    g = np.random.default_rng(25)
    N, M, K = 300, 140, 260

    def powers(*shape):
        return dev(2.0 ** g.integers(0, 4, shape) * g.integers(-1, 2, shape))

    x, x2, w, w2, dy = powers(N, K), powers(N, K), powers(M, K), powers(M, K), powers(N, M)

    def value(x, w):
        y = q.F8Matrix.quantize(w).linear(x)
        return float((dy.double() * y.double()).sum())

    size = float((dy.double().abs() * (8.0 * K * 8.0)).sum())
    tol = size * (4 * 2.0 ** -23 + 2 * (K + N) * 2.0 ** -24)
    dx = q.F8Matrix.quantize(w).transposed().gemm(q.f8_quantize(dy))
    dw = q.f8_wgrad(q.f8_quantize_t(dy), q.f8_quantize_t(x))
    assert abs(value(x2, w) - value(x, w) - float((dx.double() * (x2 - x).double()).sum())) < tol
    assert abs(value(x, w2) - value(x, w) - float((dw.double() * (w2 - w).double()).sum())) < tol
    # the values are exact up to that: each is the sum of its integers
    assert float((dx.double() - dy.double() @ w.double()).abs().max()) < 64.0 * M * (2.0 ** -22 + M * 2.0 ** -24)
    assert float((dw.double() - dy.double().t() @ x.double()).abs().max()) < 64.0 * N * (2.0 ** -22 + N * 2.0 ** -24)


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("N,S,E,M,K", [(1, 1, 1, 5, 7), (40, 2, 4, 70, 130), (300, 3, 6, 33, 140), (2, 8, 64, 24, 40),
                                       (600, 2, 2, 128, 128)])
def test_expert_gradients(N, S, E, M, K, per_slot):
    g = np.random.default_rng([24, N, E])
    ids = g.integers(0, E, (N, S)).astype(np.int32)
    if N > 1:
        ids[g.random((N, S)) < 0.2] = -1
        ids[ids == E - 1] = 0        # an expert without pairs
        ids[1, 0] = E + 3            # names no expert: no part in any gradient
    x = dev(g.standard_normal((N, S, K) if per_slot else (N, K)), torch.bfloat16)
    dy = dev(g.standard_normal((N, S, M)), torch.bfloat16)
    plan = q.route_plan(dev_u8(ids), E)
    dw = torch.full((E, M, K), float("nan"), device="cuda", dtype=DTYPES["f32" if per_slot else "bf16"])
    q.f8_wgrad(q.f8_quantize_t(dy, plan), q.f8_quantize_t(x, plan), plan, out=dw)
    xv, gv = host64(x), host64(dy)
    for e in range(E):
        t, s = np.nonzero(ids == e)
        if not len(t):
            assert bool((dw[e] == 0).all())
            continue
        rows = xv[t, s] if per_slot else xv[t]
        a = O.rows_values(*O.quantize_rows(gv[t, s].T), len(t))
        b = O.rows_values(*O.quantize_rows(rows.T), len(t))
        check(dw[e], a @ b.T, bounds(a, b), f"expert {e}")


# ---- sizes at which every tile of the products is taken --------------------------------------------

def device_check(y, a, b, label=""):
    """y against a @ b^T in fp64 on the device, a [N, K] and b [M, K] the values (fp32, exact) of the operands."""
    a, b = a.double(), b.double()
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    groups = -(-a.shape[1] // 128)
    step = 128 * 2.0 ** -23 + (groups + 18) * 2.0 ** -24 + (2.0 ** -10 if y.dtype != torch.float32 else 0.0)  # product_bound
    tol = size * step + (ref.abs() + size * step) * HALF_STEP[y.dtype] + SMALLEST[y.dtype]
    # decoded values are code * scale rounded to fp32: another half step of each factor
    tol = tol + size * 2.0 ** -22
    assert bool(((y.double() - ref).abs() <= tol).all()), label


LARGE = [  # tokens, M, K: 256 x 256, 256 x 192, 128 x 128 and 128 x 64 tiles, the last with K divided too
    (4000, 4000, 300), (4090, 2500, 4000), (2000, 8000, 250), (3000, 3000, 384), (2049, 4090, 2500), (60, 5000, 4000), (700, 130, 8000),
    (24, 4200, 300), (24, 4090, 4000), (20, 300, 4500),  # 17 .. 32 tokens: tiles, few-token kernel, tiles
    (1, 2500, 300), (16, 2500, 700), (20, 1300, 260), (3, 1, 5000)]  # rows of a workgroup across a block's edge; one row


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,K", LARGE)
def test_large_products(N, M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    dt = DTYPES[dtype]
    m = q.F8Matrix.quantize(torch.randn((M, K), generator=g, device="cuda") * 0.02)
    x = torch.randn((N, K), generator=g, device="cuda").to(dt)
    t = q.f8_quantize(x)
    y = m.linear(x)
    device_check(y, t.values(), m.dequantize(), "y")
    assert torch.equal(y, m.gemm(t, out_dtype=dt)) and torch.equal(y, m.linear(x))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("N,M,K", [(300, 4000, 4000), (250, 8000, 2000), (384, 3000, 3000), (5000, 200, 130),
                                   (4000, 4090, 2500), (16300, 100, 300), (9000, 64, 1), (2300, 700, 130)])
def test_large_weight_gradients(N, M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    gt, xt = (q.f8_quantize_t(torch.randn((N, c), generator=g, device="cuda").to(DTYPES[dtype])) for c in (M, K))
    dw = q.f8_wgrad(gt, xt, dtype=DTYPES[dtype])
    device_check(dw, gt.values(), xt.values(), "dw")
    assert torch.equal(dw, q.f8_wgrad(gt, xt, dtype=DTYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,S,E,M,K", [(4500, 2, 3, 3000, 200), (1500, 2, 3, 1000, 500), (300, 1, 250, 256, 1100), (1837, 1, 137, 925, 100),
                                       (2000, 4, 4, 500, 130)])
def test_large_expert_products(N, S, E, M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    dt = DTYPES[dtype]
    m = q.F8Matrix.quantize(torch.randn((E, M, K), generator=g, device="cuda") * 0.02)
    x = torch.randn((N, K), generator=g, device="cuda").to(dt)
    ids = torch.randint(-1, E, (N, S), generator=g, device="cuda", dtype=torch.int32)
    y = m.linear_id(x, ids)
    xv = q.f8_quantize(x).values()
    assert bool((y[ids < 0] == 0).all())
    for e in range(E):
        t, s = (ids == e).nonzero(as_tuple=True)
        if len(t):
            device_check(y[t, s], xv[t], m.dequantize(e), f"expert {e}")
    assert torch.equal(y, m.linear_id(x, ids))


# ---- streams, graphs -----------------------------------------------------------------------------

def test_side_stream_order():
    g = np.random.default_rng(25)
    m, wv = weights(g, 200, 640)
    x = dev(g.standard_normal((5, 640)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = m.linear(x * 2.0) * 0.5
    side.synchronize()
    xv = O.rows_values(*O.quantize_rows(host64(x) * 2), 640)
    check(y, xv @ wv.T * 0.5, bounds(xv, wv)[0] * 0.5)


def test_graph_replays():
    g = np.random.default_rng(26)
    M, K, E = 260, 515, 6
    m, _ = weights(g, M, K)
    ex, _ = stack(g, E, M, K)
    w = dev(g.standard_normal((M, K)) * 0.02)
    mt = m.transposed()
    x1, x300 = dev(g.standard_normal((1, K))), dev(g.standard_normal((300, K)), torch.bfloat16)
    dy = dev(g.standard_normal((300, M)) * 0.01, torch.bfloat16)
    few, many = (dev_u8(g.integers(-1, E, (n, 2)).astype(np.int32)) for n in (3, 300))

    def step():
        m.update(w, transposed=mt)
        xq, xt = q.f8_quantize_pair(x300)
        gq, gt = q.f8_quantize_pair(dy)
        plan = q.route_plan(many, E)
        return [m.linear(x1), m.gemm(xq), mt.gemm(gq), q.f8_wgrad(gt, xt), ex.linear_id(x1.expand(3, K).contiguous(), few),
                ex.linear_id(x300, many), ex.gemm_id(xq, plan)]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):   # two captures: workspaces of their own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for rep in range(3):
        for graph, out in zip(graphs, outs):
            for o in out:
                o.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(eager, out):
                assert torch.equal(a, b), f"replay {rep}"
        _ = (x300.float() * 2).sum().item()


def test_calls_on_two_streams_at_once():
    """Calls of one matrix on two streams, workspaces of their own: each gives the bits it gives alone."""
    g = np.random.default_rng(28)
    m, _ = weights(g, 512, 9728)
    xs = [dev(g.standard_normal((n, 9728)), torch.bfloat16) for n in (48, 200)]
    alone = [m.linear(x).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(s):
                outs[i].append(m.linear(x))
    torch.cuda.synchronize()
    for a, out in zip(alone, outs):
        assert all(torch.equal(a, o) for o in out)


def test_new_weights_are_seen():
    """update rewrites the borrowed codes in stream order: the next product uses them."""
    g = np.random.default_rng(27)
    w = [dev(g.standard_normal((64, 200))) for _ in range(2)]
    m = q.F8Matrix.quantize(w[0])
    x = dev(g.standard_normal((3, 200)))
    first = m.linear(x).clone()
    m.update(w[1])
    second = m.linear(x)
    assert not torch.equal(first, second)
    assert torch.equal(second, q.F8Matrix.quantize(w[1]).linear(x))


# ---- offsets past 32 bits ----------------------------------------------------------------------

def test_outputs_past_32_bits():
    """More than 2^31 outputs of a product, and of a sum over slots: the last rows are those of a small call."""
    torch.manual_seed(1)
    N, M, K = 270000, 8200, 130
    m = q.F8Matrix.quantize(torch.randn(M, K, device="cuda"))
    x = torch.randn(N, K, device="cuda").bfloat16()
    y = m.linear(x)
    assert torch.equal(y[-300:], m.linear(x[-300:]))
    out = q.route_combine(y.view(N // 2, 2, M))
    assert torch.equal(out[-100:], q.route_combine(y[-200:].view(100, 2, M)))


def test_quantized_values_past_32_bits():
    torch.manual_seed(2)
    N, K = 1050000, 2056
    x = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
    rows, cols = q.f8_quantize_pair(x)
    last, n = q.f8_quantize(x[-128:]), N % 128
    assert torch.equal(rows.codes[-128:], last.codes) and torch.equal(rows.scales[:, -128:], last.scales)
    tail = q.f8_quantize_t(x[-n - 256:])
    assert torch.equal(cols.codes[:, -384:], tail.codes) and torch.equal(cols.scales[-3:], tail.scales)


def test_weights_past_32_bits():
    E, M, K = 128, 4100, 4352
    w = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    one = q.F8Matrix.quantize(w)
    codes = torch.zeros((E, M, K), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((E,) + tuple(one.scales.shape), device="cuda")
    codes[E - 1], scales[E - 1] = one.codes, one.scales
    m = q.F8Matrix(codes, scales, M, K, E)
    for N in (3, 100):
        x = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
        ids = torch.tensor([[E - 1, 0]], dtype=torch.int32, device="cuda").expand(N, 2).contiguous()
        y = m.linear_id(x, ids)
        ref = one.linear(x, out_dtype=torch.float32)
        assert bool((y[:, 1] == 0).all())
        size = x.double().abs() @ w.double().abs().t()   # either way's error: 2^-10 of the terms (8-bit cores), 2^-8 of the result
        assert bool(((y[:, 0].double() - ref.double()).abs() <= size * 2.0 ** -9 + ref.double().abs() * 2.0 ** -8).all())


# ---- scales whose product leaves fp32's range -----------------------------------------------------

# Operands of one of three kinds.  "small": all positive, near 2^-66, so that every output is near K 2^-132, a normal fp32,
# and the two scales near 2^-75 have a product below the smallest number.  "floor": the tokens near 2^-74, where the scale
# is 2^-80, the rows near 2^-56.  "large": columns 0 of every four have tokens near 2^74 and rows of zero, columns 1 the
# other way round, columns 2 codes of 1 .. 3 steps of 2^-9 in both, columns 3 none: the scales' product is past 2^128, the
# outputs are finite.
SCALE_KINDS = ["small", "floor", "large"]


def extreme(g, kind, N, M, K, dtype):
    u = lambda r: torch.rand((r, K), generator=g, device="cuda") / 2 + 0.5  # noqa: E731
    if kind != "large":
        a, b = (2.0 ** -66, 2.0 ** -66) if kind == "small" else (2.0 ** -74, 2.0 ** -56)
        return (u(N) * a).to(dtype), (u(M) * b).to(dtype)
    out = []
    for rows, column in ((N, 0), (M, 1)):
        t = torch.zeros((rows, K), device="cuda")
        t[:, column::4] = u(rows)[:, column::4] * 2.0 ** 74
        t[:, 2::4] = torch.randint(-3, 4, (rows, K), generator=g, device="cuda")[:, 2::4] * 2.0 ** (74 - 9 - 8.8)
        out.append(t.to(dtype))
    return out


@pytest.mark.parametrize("kind", SCALE_KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,K", [(1, 300, 515), (16, 2500, 700), (20, 300, 2560), (3, 40, 9728), (100, 130, 2560), (60, 700, 4000),
                                   (300, 4000, 260), (2049, 4090, 2500), (4090, 2500, 2500)])
def test_products_of_extreme_scales(N, M, K, dtype, kind):
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w = extreme(g, kind, N, M, K, DTYPES[dtype])
    m, t = q.F8Matrix.quantize(w), q.f8_quantize(x)
    y = m.linear(x)
    device_check(y, t.values(), m.dequantize(), kind)
    assert bool((y != 0).any()) and torch.equal(y, m.gemm(t, out_dtype=DTYPES[dtype]))


@pytest.mark.parametrize("kind", SCALE_KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(130, 257, 300), (100, 300, 16300), (2500, 700, 130), (4090, 2500, 700), (4000, 4090, 500)])
def test_weight_gradients_of_extreme_scales(M, K, N, dtype, kind):
    g = torch.Generator(device="cuda").manual_seed(M)
    dy, x = (t.t() for t in extreme(g, kind, M, K, N, DTYPES[dtype]))   # the pattern of columns lies along the tokens
    gt, xt = q.f8_quantize_t(dy.contiguous()), q.f8_quantize_t(x.contiguous())
    assert gt.transposed and xt.transposed and not q.f8_quantize(x.contiguous()).transposed
    dw = q.f8_wgrad(gt, xt, dtype=DTYPES[dtype])
    device_check(dw, gt.values(), xt.values(), kind)
    assert bool((dw != 0).any())


@pytest.mark.parametrize("kind", SCALE_KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,S,E,M,K", [(4, 8, 32, 300, 512), (40, 2, 3, 70, 4000), (300, 3, 4, 520, 700), (2000, 2, 4, 300, 260)])
def test_expert_products_of_extreme_scales(N, S, E, M, K, dtype, kind):
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w = extreme(g, kind, N, E * M, K, DTYPES[dtype])
    m, ids = q.F8Matrix.quantize(w.view(E, M, K)), torch.randint(-1, E, (N, S), generator=g, device="cuda", dtype=torch.int32)
    y, xv = m.linear_id(x, ids), q.f8_quantize(x).values()
    for e in range(E):
        t, s = (ids == e).nonzero(as_tuple=True)
        if len(t):
            device_check(y[t, s], xv[t], m.dequantize(e), f"expert {e}")
    assert bool((y[ids < 0] == 0).all())


def test_bad_scales_of_a_few_rows_stay_theirs():
    """A tile whose first sweep meets scales out of range, rows of zeros, and rows with a NaN among the others."""
    g = torch.Generator(device="cuda").manual_seed(5)
    N, M, K = 300, 260, 520
    x, w = torch.randn((N, K), generator=g, device="cuda"), torch.randn((M, K), generator=g, device="cuda")
    w[128:] *= 2.0 ** -70
    x[3] = 0.0
    x[5] *= 2.0 ** -70
    x[7, 200] = float("nan")
    m, t = q.F8Matrix.quantize(w), q.f8_quantize(x)
    y = m.gemm(t)
    keep = torch.arange(N, device="cuda") != 7
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isfinite(y[keep]).all()) and bool((y[3] == 0).all())
    device_check(y[keep], t.values()[keep], m.dequantize())
    plain = q.F8Matrix.quantize(w[:128].contiguous())   # alone, without the second sweep: within its last bits
    device_check(plain.gemm(t)[keep], t.values()[keep], plain.dequantize())


def test_dequantize_more_than_32_bits_of_threads():
    M, K = 1 << 24, 2100
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("needs 120 GB")
    codes = torch.zeros((M, 2176), dtype=torch.uint8, device="cuda")
    codes[-5:, :K] = torch.randint(0, 126, (5, K), device="cuda", dtype=torch.uint8)
    codes[3, :K] = codes[-1, :K]
    m = q.F8Matrix(codes, torch.full((M // 128, 17), 0.5, device="cuda"), M, K)
    w = m.dequantize(dtype=torch.bfloat16)
    last = codes[-5:, :K].view(torch.float8_e4m3fn).bfloat16() * 0.5
    assert torch.equal(w[-5:], last) and torch.equal(w[3], last[-1])
    assert all(bool((w[i:i + 8] == 0).all()) for i in (4, M // 2, M // 2 - 8, M - 13))
    del w, m, codes
    torch.cuda.empty_cache()


# ---- 16-bit outputs to one rounding ---------------------------------------------------------------

# Codes of -8 .. 8 and scales of 1/2, 1 and 2: products of an octet span 6 bits, which the 8-bit cores hold, a group's sum
# is a whole number below 2^13 and the sum over 32 groups of it times 1/4 .. 4 has 22 bits.  Every order of the sums is
# exact in fp32, so that an output is its exact value rounded once.

def whole_codes(g, rows, K, lead=()):
    codes = torch.zeros(lead + (rows, O.padded(K)), device="cuda")
    codes[..., :K] = torch.randint(-8, 9, lead + (rows, K), generator=g, device="cuda").float()
    return codes.to(torch.float8_e4m3fn)


def powers_of_two(g, *shape):
    return 2.0 ** torch.randint(-1, 2, shape, generator=g, device="cuda").float()


def whole_tokens(g, rows, K):
    t = q.F8Tokens(whole_codes(g, rows, K), powers_of_two(g, O.padded(K) // 128, rows), rows, K)
    return t, t.values().double()


@pytest.mark.parametrize("N,M,K", LARGE + [(32, 2000, 4096), (8, 515, 130), (300, 257, 3900)])
def test_products_to_one_rounding(N, M, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    blocks = powers_of_two(g, O.padded(M) // 128, O.padded(K) // 128)
    m = q.F8Matrix(whole_codes(g, M, K), blocks, M, K)
    t, x = whole_tokens(g, N, K)
    y = x @ m.dequantize().double().t()
    for dt in DTYPES.values():
        assert torch.equal(m.gemm(t, out_dtype=dt), y.to(dt)), dt


@pytest.mark.parametrize("N,M,K", [(300, 4000, 4000), (4000, 4090, 2500), (250, 8000, 2000), (384, 3000, 3000), (4000, 100, 300), (1000, 700, 130)])
def test_weight_gradients_to_one_rounding(N, M, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    (gt, a), (xt, b) = whole_tokens(g, M, N), whole_tokens(g, K, N)
    dw = a @ b.t()
    for dt in DTYPES.values():
        assert torch.equal(q.f8_wgrad(gt, xt, dtype=dt), dw.to(dt)), dt


@pytest.mark.parametrize("N,S,E,M,K", [(4500, 2, 3, 3000, 200), (1500, 2, 3, 1000, 500), (300, 1, 250, 256, 1100), (2000, 4, 4, 500, 130),
                                       (40, 2, 8, 64, 4000)])
def test_expert_products_to_one_rounding(N, S, E, M, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    m = q.F8Matrix(whole_codes(g, M, K, (E,)), powers_of_two(g, E, O.padded(M) // 128, O.padded(K) // 128), M, K, E)
    t, x = whole_tokens(g, N, K)
    ids = torch.randint(-1, E, (N, S), generator=g, device="cuda", dtype=torch.int32)
    plan = q.route_plan(ids, E)
    for dt in DTYPES.values():
        y = m.gemm_id(t, plan, out_dtype=dt)
        for e in range(E):
            n, s = (ids == e).nonzero(as_tuple=True)
            assert torch.equal(y[n, s], (x[n] @ m.dequantize(e).double().t()).to(dt)), (e, dt)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 16, 300, 2049])
def test_a_channel_300_times_larger(N, dtype):
    """Hidden states have such channels: their octet's other products lose bits on the 8-bit cores, within the bound."""
    g = torch.Generator(device="cuda").manual_seed(N)
    M, K = 1000, 2560
    x = torch.randn((N, K), generator=g, device="cuda")
    x[:, 77] *= 300.0
    m, t = q.F8Matrix.quantize(torch.randn((M, K), generator=g, device="cuda") * 0.02), q.f8_quantize(x)
    y = m.gemm(t, out_dtype=DTYPES[dtype])
    device_check(y, t.values(), m.dequantize(), "channel")
    # beside the output's own rounding the cores cost less than 2^-13 of the root mean square, the cut of the largest products
    ref = t.values().double() @ m.dequantize().double().t()
    own, all_ = ((v.double() - ref).pow(2).mean().sqrt() / ref.pow(2).mean().sqrt() for v in (ref.to(y.dtype), y))
    assert float(all_) ** 2 <= float(own) ** 2 * 1.02 + 2.0 ** -26


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,K", [(300, 260, 520), (2049, 4090, 300), (60, 700, 4000)])
def test_blocks_of_zeros_and_of_small_values(N, M, K, dtype):
    """Zero rows against zero blocks, beside rows and blocks of ordinary, of small and of the smallest values."""
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w = torch.randn((N, K), generator=g, device="cuda"), torch.randn((M, K), generator=g, device="cuda")
    x[::3] = 0.0
    x[1::7] *= 2.0 ** -90
    x[2::11] *= 2.0 ** -62
    w[:128] = 0.0
    w[128:256] *= 2.0 ** -90
    w[256:] *= 2.0 ** -62
    x, w = x.to(DTYPES[dtype]), w.to(DTYPES[dtype])
    m, t = q.F8Matrix.quantize(w), q.f8_quantize(x)
    y = m.gemm(t, out_dtype=DTYPES[dtype])
    assert bool((y[::3] == 0).all()) and bool((y[:, :128] == 0).all())
    a, b = t.values(), m.dequantize()
    ref, size = a.double() @ b.double().t(), a.double().abs() @ b.double().abs().t()
    groups = -(-K // 128)
    tol = size * (2.0 ** -10 + 2.0 ** -21) + (ref.abs() + size * 2.0 ** -9) * HALF_STEP[y.dtype] + SMALLEST[y.dtype] + groups * 2.0 ** -135
    assert bool(((y.double() - ref).abs() <= tol).all())


def test_a_copy_outlives_its_matrix():
    import copy
    g = torch.Generator(device="cuda").manual_seed(6)
    m = q.F8Matrix.quantize(torch.randn((3, 70, 200), generator=g, device="cuda"))
    x = torch.randn((5, 200), generator=g, device="cuda")
    ids = torch.randint(0, 3, (5, 2), generator=g, device="cuda", dtype=torch.int32)
    y = m.linear_id(x, ids)
    twin, third = copy.copy(m), copy.copy(m)
    del third
    assert torch.equal(m.linear_id(x, ids), y)
    m.close()
    assert torch.equal(twin.linear_id(x, ids), y) and twin.codes is m.codes
    with pytest.raises(q.QmmError, match="handle"):
        m.linear_id(x, ids)


@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,K", [(1, 130, 300), (20, 300, 700), (130, 257, 300), (2500, 700, 130), (4090, 2500, 700), (4000, 4090, 500), (100, 300, 16300)])
def test_one_operand_past_2_100(N, M, K, dtype, swap):
    """Values near 2^114 against values near 2^-40, of one sign: a group's sum times the larger scale alone overflows."""
    g = torch.Generator(device="cuda").manual_seed(N)
    a, b = (((torch.rand((rows, K), generator=g, device="cuda") / 4 + 0.75) * s).to(DTYPES[dtype])
            for rows, s in ((N, 2.0 ** (-40 if swap else 114)), (M, 2.0 ** (114 if swap else -40))))
    m, t = q.F8Matrix.quantize(b), q.f8_quantize(a)
    device_check(m.gemm(t, out_dtype=DTYPES[dtype]), t.values(), m.dequantize(), "product")
    gt, xt = q.f8_quantize_t(a.t().contiguous()), q.f8_quantize_t(b.t().contiguous())
    device_check(q.f8_wgrad(gt, xt, dtype=DTYPES[dtype]), gt.values(), xt.values(), "weight gradient")
