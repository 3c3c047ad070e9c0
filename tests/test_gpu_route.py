"""The expert router, balance loss, their gradients and the sum of the slots, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import block_quantized_weight_matmul_amd as q
from oracle import f8 as F8
from oracle import route as O
from tests.gpu_helpers import to_host
from tests.test_gpu_f8 import DTYPES, HALF_STEP, check, dev, dev_u8, host64, id_reference, quantized_values, stack

pytestmark = pytest.mark.gpu

# relative error of a probability: the difference l - max is exact to half a step (at most 2^-24 * |l - max|, |l - max|
# below 64 here where p matters: 2^-18), expf within 2 steps, sums of up to 1024 terms, a quotient
P_REL = 2.0 ** -18 + 4 * 2.0 ** -23 + 1024 * 2.0 ** -24


def logits_of(g, N, E, dtype, masked=0.0):
    l = g.standard_normal((N, E)) * 2
    l[g.random((N, E)) < masked] = -np.inf
    if masked and N > 2:
        l[N // 2] = -np.inf
    return dev(l, DTYPES[dtype])


def compare(r, want, N, label=""):
    assert np.array_equal(to_host(r.ids), want["ids"]), f"{label}: ids"
    assert np.array_equal(to_host(r.counts), want["counts"]), f"{label}: counts"
    tol = P_REL * (N + 1)
    assert np.allclose(host64(r.weights), want["weights"], rtol=2 * P_REL, atol=1e-30, equal_nan=True), f"{label}: weights"
    assert np.allclose(host64(r.psum), want["psum"], rtol=P_REL + N * 2.0 ** -24, atol=1e-30, equal_nan=True), f"{label}: psum"
    assert np.allclose(host64(r.loss), want["loss"], rtol=tol, equal_nan=True), f"{label}: loss"


SIZES = [(1, 1, 1), (1, 4, 2), (16, 128, 8), (33, 8, 2), (100, 60, 6), (64, 16, 16), (5, 17, 3), (7, 200, 64),
         (300, 256, 8), (20, 500, 10), (3, 1000, 64), (9, 1024, 8), (9, 1023, 1), (5000, 64, 4),
         (37, 201, 3), (37, 203, 4), (300, 399, 7), (37, 402, 12), (140, 402, 20), (37, 777, 5), (130, 513, 2)]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,E,S", SIZES)
def test_route(N, E, S, dtype):
    g = np.random.default_rng([31, N, E])
    for normalise in (False, True):
        l = logits_of(g, N, E, dtype, 0.2 if normalise else 0.0)
        r = q.route(l, S, normalise=normalise, coef=0.01)
        want = O.route(host64(l), S, normalise, 0.01)
        compare(r, want, N, f"normalise {normalise}")
        again = q.route(l, S, normalise=normalise, coef=0.01)
        assert all(torch.equal(a, b) for a, b in zip(r[:5], again[:5])), "two calls, two results"
        loss = q.balance_loss(r.counts, r.psum, S, 0.01)
        assert np.isclose(host64(loss), want["loss"], rtol=P_REL * (N + 1))


def test_ties_go_to_the_lower_index():
    for E in (8, 40, 300):
        l = torch.zeros((3, E), device="cuda", dtype=torch.bfloat16)
        l[1, E - 2:] = 1.0
        l[2, ::2] = -0.0
        r = q.route(l, 4)
        assert r.ids.tolist()[0] == [0, 1, 2, 3] and r.ids.tolist()[1] == [E - 2, E - 1, 0, 1]
        assert r.ids.tolist()[2] == [0, 1, 2, 3]


@pytest.mark.parametrize("S", [3, 8, 17, 40])
@pytest.mark.parametrize("E", [70, 131, 250, 500, 1000])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_order_of_extreme_logits(dtype, E, S):
    """The largest and lowest numbers, subnormal ones, both zeros and close neighbours, each several times, in any place."""
    g = np.random.default_rng([32, E, S])
    t = DTYPES[dtype]
    top, tiny = torch.finfo(t).max, float(torch.finfo(t).smallest_normal)
    step = float(torch.finfo(t).eps)
    some = [top, -top, top / 2, -top / 2, tiny, -tiny, tiny * step, -tiny * step, 0.0, -0.0, 1.0, 1.0 + step, -1.0, -1.0 - step, -np.inf]
    l = dev(g.choice(some, (60, E)), t)
    got = to_host(q.route(l, S).ids)
    v = host64(l)
    order = np.argsort(-v, axis=1, kind="stable")[:, :S]
    want = np.where(np.take_along_axis(v, order, 1) > -np.inf, order, -1)
    assert np.array_equal(got, want)


def test_masks_that_leave_little():
    inf = float("inf")
    l = torch.tensor([[-inf, -inf, -inf, -inf], [-inf, 1.0, -inf, -inf], [0.0, 1.0, 2.0, 3.0],
                      [torch.finfo(torch.float32).min] * 4], device="cuda")
    for normalise in (False, True):
        r = q.route(l, 3, normalise=normalise, coef=1.0)
        compare(r, O.route(host64(l), 3, normalise, 1.0), 4)
        d = q.route_backward(l, r, torch.ones((4, 3), device="cuda"), torch.ones((), device="cuda"))
        assert bool((d[0] == 0).all()) and bool(torch.isfinite(d).all())
    empty = torch.full((5, 4), -inf, device="cuda")
    r = q.route(empty, 2, coef=1.0)
    assert bool((r.ids == -1).all()) and bool((r.weights == 0).all()) and bool((r.counts == 0).all())
    assert r.loss.item() == 0.0 and bool((r.psum == 0).all())
    assert bool((q.route_backward(empty, r, torch.ones((5, 2), device="cuda"), torch.ones((), device="cuda")) == 0).all())


def test_nan_and_infinite_logits_are_loud():
    l = torch.randn((4, 10), device="cuda")
    l[1, 3] = float("nan")
    l[2, 5] = float("inf")
    for normalise in (False, True):
        r = q.route(l, 2, normalise=normalise, coef=1.0)
        assert bool(torch.isnan(r.weights[1]).all()) and bool(torch.isnan(r.weights[2]).all())
        assert bool(torch.isfinite(r.weights[0]).all()) and bool(torch.isfinite(r.weights[3]).all())
        assert 3 not in r.ids[1].tolist() and r.ids[2, 0].item() == 5
        assert torch.isnan(r.loss)


def test_padded_rows():
    g = np.random.default_rng(32)
    l = logits_of(g, 50, 32, "bf16")
    valid = dev_u8((g.random(50) < 0.7).astype(np.uint8))
    for v in (valid, valid.bool()):
        r = q.route(l, 4, coef=0.1, valid=v)
        want = O.route(host64(l), 4, True, 0.1, to_host(valid))
        compare(r, want, 50)
        dw = dev(g.standard_normal((50, 4)))
        d = q.route_backward(l, r, dw, torch.ones((), device="cuda"))
        assert bool((d[~valid.bool()] == 0).all())
        ref = O.route_backward(host64(l), want, True, 0.1, host64(dw), 1.0)
        assert_gradient(d, ref, want, host64(dw), True, 0.1)


def test_no_rows():
    l = torch.empty((0, 12), device="cuda")
    r = q.route(l, 3, coef=1.0)
    assert r.ids.shape == (0, 3) and bool((r.counts == 0).all()) and bool((r.psum == 0).all()) and r.loss.item() == 0
    assert q.route_backward(l, r, torch.empty((0, 3), device="cuda")).shape == (0, 12)
    assert bool((q.route_plan(r.ids, 12).counts == 0).all())


def assert_gradient(d, ref, want, dw, normalise, dloss_coef):
    """p (dp - sum p dp): every factor is off by P_REL at most, so the bound is that of the sums of magnitudes."""
    T = max(int(want["counts"][-1]), 1)
    E = ref.shape[1]
    S = want["ids"].shape[1]
    f = want["counts"][:E] * E / (S * T)
    k = want["ids"] >= 0
    size = np.abs(dloss_coef * f / T)[None, :] * np.ones_like(ref)
    chosen = np.where(k, np.take_along_axis(want["p"], np.maximum(want["ids"], 0), 1), 0)
    total = np.where(chosen.sum(1) > 0, chosen.sum(1), 1)[:, None] if normalise else 1.0
    adw = np.where(k, np.abs(dw), 0)
    part = (adw + (adw * want["weights"]).sum(1, keepdims=True)) / total if normalise else adw
    for t in range(ref.shape[0]):
        size[t, want["ids"][t][k[t]]] += part[t][k[t]]
    bound = want["p"] * (size + (want["p"] * size).sum(1, keepdims=True)) * (6 * P_REL + E * 2.0 ** -23)
    check(d, ref, bound + 1e-37, "dlogits")


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,E,S", [(1, 4, 2), (1, 1, 1), (33, 8, 2), (16, 128, 8), (100, 60, 6), (7, 200, 64), (300, 256, 8),
                                   (9, 1024, 8)])
def test_route_backward(N, E, S, dtype):
    g = np.random.default_rng([33, N, E])
    for normalise in (False, True):
        l = logits_of(g, N, E, dtype, 0.2 if normalise else 0.0)
        dw = dev(g.standard_normal((N, S)))
        r = q.route(l, S, normalise=normalise, coef=0.05)
        want = O.route(host64(l), S, normalise, 0.05)
        for use_w, dloss in ((True, 1.5), (True, None), (False, 1.5), (False, None)):
            d = q.route_backward(l, r, dw if use_w else None, torch.tensor(dloss, device="cuda") if dloss else None)
            assert d.dtype == l.dtype
            ref = O.route_backward(host64(l), want, normalise, 0.05, host64(dw) if use_w else None, dloss)
            assert_gradient(d, ref, want, host64(dw) * use_w, normalise, 0.05 * (dloss or 0.0))


def test_backward_against_differences():
    """The device's own forward, differenced: weights are smooth where the chosen set does not change."""
    g = np.random.default_rng(34)
    N, E, S, h = 6, 12, 3, 2.0 ** -6
    l = dev(np.round(g.standard_normal((N, E)) * 64) / 16)
    dw = dev(g.standard_normal((N, S)))
    for normalise in (False, True):
        r = q.route(l, S, normalise=normalise, coef=0.5)
        d = host64(q.route_backward(l, r, dw, torch.ones((), device="cuda")))
        f = host64(r.counts)[:E] * E / (S * N)
        value = lambda x: ((host64(dw) * host64(x.weights)).sum() + 0.5 * (f * host64(x.psum)).sum() / N)  # noqa: E731
        for t in range(N):
            for e in range(E):
                up, down = l.clone(), l.clone()
                up[t, e] += h
                down[t, e] -= h
                a, b = (q.route(x, S, normalise=normalise, coef=0.5) for x in (up, down))
                if not (torch.equal(a.ids, r.ids) and torch.equal(b.ids, r.ids)):
                    continue
                # third derivatives of these are below 16 in sum: h^2 / 6 of them, and the forward's error over 2 h
                assert abs((value(a) - value(b)) / (2 * h) - d[t, e]) < 16 * h * h / 6 + 1e-4


@pytest.mark.parametrize("normalise", [False, True])
def test_counts_summed_over_parts_of_a_batch(normalise):
    """A batch in three parts: loss and gradients from the summed counts and probabilities are those of the whole."""
    g = np.random.default_rng(39)
    N, E, S, coef = 300, 40, 3, 0.02
    l = logits_of(g, N, E, "f32", 0.1)
    dw, dloss = dev(g.standard_normal((N, S))), torch.full((1,), 2.0, device="cuda")
    whole = q.route(l, S, normalise=normalise, coef=coef)
    cuts = (0, 70, 71, N)
    parts = [q.route(l[a:b], S, normalise=normalise, coef=coef) for a, b in zip(cuts, cuts[1:])]
    counts = sum(p.counts for p in parts)
    psum = sum(p.psum for p in parts)
    assert torch.equal(counts, whole.counts)
    want = O.route(host64(l), S, normalise, coef)
    assert np.isclose(host64(q.balance_loss(counts, psum, S, coef)), want["loss"], rtol=P_REL * (N + 1))
    d = q.route_backward(l, whole, dw, dloss)
    for (a, b), p in zip(zip(cuts, cuts[1:]), parts):
        assert torch.equal(p.ids, whole.ids[a:b]) and torch.equal(p.weights, whole.weights[a:b])
        assert torch.equal(q.route_backward(l[a:b], p._replace(counts=counts), dw[a:b], dloss), d[a:b])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("N,S,M", [(1, 1, 1), (3, 2, 7), (5, 8, 520), (64, 3, 1024), (2, 64, 100), (1000, 2, 24)])
def test_combine(N, S, M, dtype):
    g = np.random.default_rng([35, N, S])
    dt = DTYPES[dtype]
    y, dout = dev(g.standard_normal((N, S, M)), dt), dev(g.standard_normal((N, M)), dt)
    yv, dv = host64(y), host64(dout)
    check(q.route_combine(y), O.combine(yv), np.abs(yv).sum(1) * S * 2.0 ** -24, "sum")
    for wt in {torch.float32, dt}:
        w = dev(g.random((N, S)), wt)
        wv = host64(w)
        check(q.route_combine(y, w), O.combine(yv, wv), O.combine(np.abs(yv), wv) * S * 2.0 ** -24, "weighted")
        dy, dw = q.route_combine_backward(y, w, dout)
        assert dy.dtype == dt and dw.dtype == wt
        check(dy, wv[:, :, None] * dv[:, None, :], np.abs(wv[:, :, None] * dv[:, None, :]) * 2.0 ** -24, "dy")
        check(dw, (yv * dv[:, None, :]).sum(2), (np.abs(yv) * np.abs(dv)[:, None, :]).sum(2) * (M + 64) * 2.0 ** -24, "dw")


def test_combine_against_differences():
    """<dout, combine> is linear in y and in the weights: one step each, of whole numbers, is exact."""
    g = np.random.default_rng(40)
    N, S, M = 20, 3, 33
    y, y2, dout = dev(g.integers(-8, 9, (N, S, M))), dev(g.integers(-8, 9, (N, S, M))), dev(g.integers(-4, 5, (N, M)))
    w, w2 = dev(g.integers(-4, 5, (N, S))), dev(g.integers(-4, 5, (N, S)))

    def value(y, w):
        return float((q.route_combine(y, w).double() * dout.double()).sum())

    dy, dw = q.route_combine_backward(y, w, dout)
    assert value(y2, w) - value(y, w) == float((dy.double() * (y2 - y).double()).sum())
    assert value(y, w2) - value(y, w) == float((dw.double() * (w2 - w).double()).sum())


def test_unaligned_views():
    g = np.random.default_rng(36)
    buf = dev(g.standard_normal(3 * 2 * 16 + 1), torch.float16)
    y = buf[1:].view(3, 2, 16)
    w = torch.rand((3, 2), device="cuda")
    assert torch.equal(q.route_combine(y, w), q.route_combine(y.clone(), w))
    l = dev(g.standard_normal(4 * 128 + 1))[1:].view(4, 128)
    a, b = q.route(l, 8), q.route(l.clone(), 8)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)
    ones = torch.ones((4, 8), device="cuda")
    assert torch.equal(q.route_backward(l, a, ones), q.route_backward(l.clone(), b, ones))


def test_router_experts_and_gradients_together():
    """A router, its experts' e4m3 products, the weighted sum, and every gradient, as a training step uses them."""
    g = np.random.default_rng(37)
    N, E, S, M, K = 150, 12, 3, 96, 200
    experts, values = stack(g, E, M, K)
    x = dev(g.standard_normal((N, K)))
    l = logits_of(g, N, E, "f32", 0.1)
    dout = dev(g.standard_normal((N, M)) * 0.1)
    r = q.route(l, S, coef=0.01)
    plan = q.route_plan(r.ids, E)
    assert torch.equal(plan.counts, r.counts[:E])
    y = experts.gemm_id(q.f8_quantize(x), plan)
    out = q.route_combine(y, r.weights)
    dy, dweights = q.route_combine_backward(y, r.weights, dout)
    dx = q.route_combine(experts.transposed().gemm_id(q.f8_quantize(dy.view(N * S, M)), plan))
    dw = q.f8_wgrad(q.f8_quantize_t(dy, plan), q.f8_quantize_t(x, plan), plan)
    dlogits = q.route_backward(l, r, dweights, torch.ones((), device="cuda"))

    want = O.route(host64(l), S, True, 0.01)
    ids = want["ids"]
    yv, (bound, _) = id_reference(quantized_values(x), ids, values, M)
    w = host64(r.weights)
    check(out, O.combine(yv, w), O.combine(bound + np.abs(yv) * (S + 1) * 2.0 ** -24, w), "out")
    dv = host64(dout)
    yd = host64(y)
    check(dweights, (yd * dv[:, None, :]).sum(2), (np.abs(yd) * np.abs(dv)[:, None, :]).sum(2) * M * 2.0 ** -23, "dweights")
    gq = quantized_values(dy)
    dref, dbound = np.zeros((N, S, K)), np.zeros((N, S, K))
    for e in range(E):
        t, s = np.nonzero(ids == e)
        if len(t):
            dref[t, s] = gq[t, s] @ values[e]
            dbound[t, s] = F8.product_bound(gq[t, s], values[e].T)
            a = F8.rows_values(*F8.quantize_rows(host64(dy)[t, s].T), len(t))
            b = F8.rows_values(*F8.quantize_rows(host64(x)[t].T), len(t))
            check(dw[e], a @ b.T, F8.product_bound(a, b), f"dw {e}")
        else:
            assert bool((dw[e] == 0).all())
    dbound += np.abs(dref) * HALF_STEP[torch.float32]
    check(dx, dref.sum(1), dbound.sum(1) + np.abs(dref).sum(1) * S * 2.0 ** -24, "dx")
    ref = O.route_backward(host64(l), want, True, 0.01, host64(dweights), 1.0)
    assert_gradient(dlogits, ref, want, host64(dweights), True, 0.01)


def test_route_in_graph():
    g = np.random.default_rng(38)
    l = logits_of(g, 700, 64, "bf16", 0.1)
    dw = dev(g.standard_normal((700, 4)))
    one = torch.ones((), device="cuda")

    def step():
        r = q.route(l, 4, coef=0.01)
        return [r.ids, r.weights, r.counts, r.psum, r.loss, q.route_backward(l, r, dw, one), q.route_plan(r.ids, 64).counts]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)), rep
        _ = l.float().clamp(min=-10).sum().item()


def test_logits_past_32_bits():
    """More than 2^31 logits: the last rows, and their gradients, are those of a small call."""
    N, E, S = 2100000, 1023, 2
    l = torch.randn(N, E, device="cuda", dtype=torch.bfloat16)
    r, few = q.route(l, S), q.route(l[-50:], S)
    assert torch.equal(r.ids[-50:], few.ids) and torch.equal(r.weights[-50:], few.weights)
    assert int(r.counts[:E].long().sum()) == N * S and int(r.counts[E]) == N
    dw = torch.randn(N, S, device="cuda")
    d = q.route_backward(l, r, dw)
    assert torch.equal(d[-50:], q.route_backward(l[-50:], few, dw[-50:]))


@pytest.mark.parametrize("tiled", [False, True])
def test_router_ids_through_the_block_formats(tiled):
    """The router's ids go into the block formats' expert products, where an id of -1 makes a NaN row: its weight is 0, and
    the sum leaves the slot out.  Backward, an empty slot has no gradient."""
    g = np.random.default_rng(41)
    N, E, S, M, K = 24, 5, 3, 64, 512
    values = g.standard_normal((E, M, K)).astype(np.float32) * 0.05
    blocks = torch.cat([q.quantize(dev(v), "q8_0").view(-1) for v in values])
    experts = q.QMatrix(blocks, "q8_0", M, K, E)
    l = logits_of(g, N, E, "f32", 0.5)
    r = q.route(l, S, coef=0.01)
    assert bool((r.ids == -1).any()) and int(r.counts[E]) < N
    x, dout = dev(g.standard_normal((N, K))), dev(g.standard_normal((N, M)))
    y = (experts.gemm_id_tiled if tiled else experts.gemm_id)(x, r.ids)
    empty = r.ids == -1
    assert bool(torch.isnan(y[empty]).all()) and bool((r.weights[empty] == 0).all())
    w = host64(r.weights)
    for dt in DTYPES.values():
        yt = y.to(dt)
        yv = np.where(to_host(empty)[:, :, None], 0, host64(yt))
        check(q.route_combine(yt, r.weights), O.combine(yv, w), O.combine(np.abs(yv), w) * S * 2.0 ** -24, f"out {dt}")
    dy, dw = q.route_combine_backward(y, r.weights, dout)
    assert bool((dy[empty] == 0).all())
    d = q.route_backward(l, r, dw, torch.ones((), device="cuda"))
    want = O.route(host64(l), S, True, 0.01)
    dwv = np.where(to_host(empty), 0, host64(dw))
    assert_gradient(d, O.route_backward(host64(l), want, True, 0.01, dwv, 1.0), want, dwv, True, 0.01)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("M", [5, 24])
def test_slots_of_weight_zero_add_nothing(dtype, M):
    dt = DTYPES[dtype]
    y = torch.ones((3, 2, M), device="cuda", dtype=dt)
    y[0, 1], y[1, 0], y[2] = float("nan"), float("inf"), float("nan")
    for wt in {torch.float32, dt}:
        w = torch.tensor([[2.0, 0.0], [-0.0, 3.0], [0.0, 0.0]], device="cuda", dtype=wt)
        out = q.route_combine(y, w)
        assert out[:, 0].tolist() == [2.0, 3.0, 0.0] and torch.equal(out, out[:, :1].expand(3, M))
        w[1, 0] = float("nan")      # a NaN weight stays one
        assert bool(torch.isnan(q.route_combine(y, w)[1]).all())
    assert bool(torch.isnan(q.route_combine(y)[0]).all())   # a plain sum has every slot


def test_sums_of_the_most_tokens():
    """2^24 tokens: as many workgroups of 256 threads as HIP takes no longer along one axis."""
    N = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(1)
    y, dout = (torch.randn((N, 1, 1), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand((N, 1), generator=g, device="cuda")
    dy, dw = q.route_combine_backward(y, w, dout[:, 0])
    assert torch.equal(dy, (w[:, :, None] * dout.float()).bfloat16()) and torch.equal(dw, (y.float() * dout.float())[:, 0])
    assert torch.equal(q.route_combine(y, w), (w[:, :, None] * y.float()).bfloat16()[:, 0])


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB")


def test_sums_of_more_than_32_bits_of_threads():
    N, M = 1 << 24, 2056
    room(150)
    y, w = torch.zeros((N, 1, M), device="cuda", dtype=torch.bfloat16), torch.full((N, 1), 2.0, device="cuda")
    y[-3:] = torch.randn((3, 1, M), device="cuda")
    y[5] = torch.randn((1, M), device="cuda")
    out = torch.full((N, M), 7.0, device="cuda", dtype=torch.bfloat16)
    q.route_combine(y, w, out=out)
    assert torch.equal(out[-3:], 2 * y[-3:, 0]) and torch.equal(out[5], 2 * y[5, 0])
    assert all(bool((out[i:i + 8] == 0).all()) for i in (6, 1 << 23, (1 << 23) - 8, N - 11))
    del y, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,S", [(16, 3), (128, 8), (600, 20)])
def test_more_rows_than_one_pass(E, S, dtype):
    """40000 rows are two or more for each of a launch's teams of lanes: what a team carries from row to row (sums, a row of
    LDS with the loss's gradient) is right after the first.  Ids, weights and gradients are those of calls on 4000 rows,
    which are one a team, bit for bit; the sums are those of fp64."""
    g = np.random.default_rng([42, E])
    N, coef, part = 40000, 0.03, 4000
    l = logits_of(g, N, E, dtype, 0.1)
    valid = dev_u8((g.random(N) < 0.9).astype(np.uint8))
    dw, dloss = dev(g.standard_normal((N, S))), torch.full((), 1.5e4, device="cuda")
    for normalise in (False, True):
        r = q.route(l, S, normalise=normalise, coef=coef, valid=valid)
        counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        d = q.route_backward(l, r, dw, dloss)
        loss_only = q.route_backward(l, r, None, dloss)
        for a in range(0, N, part):
            s = slice(a, a + part)
            p = q.route(l[s], S, normalise=normalise, coef=coef, valid=valid[s])
            assert torch.equal(p.ids, r.ids[s]) and torch.equal(p.weights, r.weights[s])
            counts += p.counts
            p = p._replace(counts=r.counts)
            assert torch.equal(q.route_backward(l[s], p, dw[s], dloss), d[s]), a
            assert torch.equal(q.route_backward(l[s], p, None, dloss), loss_only[s]), a
        assert torch.equal(counts, r.counts.long()) and bool((loss_only != 0).any())
        alive = (l > -float("inf")).any(1) & valid.bool()
        assert int(alive.sum()) == int(r.counts[E])
        psum = to_host(torch.softmax(l[alive].double(), 1).sum(0))
        assert np.allclose(host64(r.psum), psum, rtol=P_REL + N * 2.0 ** -24)
        want = O.balance_loss(to_host(r.counts).astype(np.int64), psum, S, coef)
        assert np.isclose(host64(r.loss), want, rtol=P_REL + N * 2.0 ** -24 + (E + 8) * 2.0 ** -23)
