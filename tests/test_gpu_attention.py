"""Head norms and rotation, the paged cache and attention on the device, against the fp64 oracle."""

import copy

import numpy as np
import pytest
import torch

import block_quantized_weight_matmul_amd as q
from oracle import attention as A
from tests.gpu_helpers import to_host
from tests.test_gpu_f8 import DTYPES, HALF_STEP, SMALLEST, dev, host64

pytestmark = pytest.mark.gpu

EPS = 1e-6
HALF = {"f16": torch.float16, "bf16": torch.bfloat16}


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def within(y, ref, bound, label=""):
    """|y - ref| <= bound plus half a step of y's type."""
    got = host64(y)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    tol = bound + (np.abs(ref) + bound) * HALF_STEP[y.dtype] + SMALLEST[y.dtype]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{label}: {bad.sum()} of {got.size}; worst {np.nanmax(np.abs(got - ref) / tol)} of the bound"


# ---- norms and rotation ------------------------------------------------------------------------

# Relative error of a normed value before its last rounding, in units of 2^-24: the sum of up to 256 squares in chains of 8
# and a tree of 5 levels (13 roundings, halved by the root), its mean and eps (2, halved), root, quotient and two products
# (4).  A rotation adds the cosine's rounding, a product's and a sum's (3).
HEAD_REL = (6.5 + 1 + 4 + 3) * 2.0 ** -24


def frequencies(R):
    return (1e6 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)


def head_inputs(g, T, Hq, H, D, dtype, strided):
    if strided:  # slices of one projection's output, three columns further for rows that start anywhere
        rows = dev(g.standard_normal((T, (Hq + 2 * H) * D + 3)) * 2, dtype)
        rows = rows[:, 3:].unflatten(1, (Hq + 2 * H, D))
        return rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
    return tuple(dev(g.standard_normal((T, n, D)) * 2, dtype) for n in (Hq, H, H))


HEADS = [(1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (3, 5, 2, 80, 48), (7, 4, 4, 64, 64), (70, 15, 5, 96, 64), (5, 3, 1, 256, 256),
         (33, 6, 2, 144, 8), (9, 2, 2, 32, 32), (5000, 2, 1, 128, 64), (130, 16, 8, 112, 112)]


@pytest.mark.parametrize("x,out", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,Hq,H,D,R", HEADS)
def test_norm_and_rotation(T, Hq, H, D, R, x, out):
    g = np.random.default_rng([71, T, D, R])
    for interleaved in (False, True):
        qx, kx, _ = head_inputs(g, T, Hq, H, D, DTYPES[x], interleaved)
        qw, kw = (1 + 0.2 * g.standard_normal((2, D))).astype(np.float32)
        pos = g.integers(0, 1 << 20, T)
        pos[-1] = (1 << 31) - 1
        freq = frequencies(R)
        got = q.head_norm_rope(qx, kx, i32(pos), dev(freq), dev(qw), dev(kw), eps=EPS, interleaved=interleaved, dtype=DTYPES[out])
        for y, src, w in zip(got, (qx, kx), (qw, kw)):
            ref, size = A.heads(host64(src), w, EPS, pos, freq, interleaved)
            assert y.is_contiguous()
            within(y, ref, size * HEAD_REL, f"interleaved {interleaved}")


def test_norm_alone_and_rotation_alone():
    g = np.random.default_rng(72)
    T, D = 17, 64
    qx, kx, _ = head_inputs(g, T, 4, 2, D, torch.float32, False)
    w, pos, freq = (1 + g.random(D)).astype(np.float32), g.integers(-50, 5000, T), frequencies(D)
    for dtype in DTYPES.values():  # weights of any type
        wd = dev(w, dtype)
        a, b = q.head_norm_rope(qx, kx, None, None, wd, wd)
        for y, src in ((a, qx), (b, kx)):
            ref, size = A.heads(host64(src), host64(wd), 1e-6, None, None, False)
            within(y, ref, size * HEAD_REL)
    a, b = q.head_norm_rope(qx, kx, i32(pos), dev(freq))
    for y, src in ((a, qx), (b, kx)):
        ref, size = A.heads(host64(src), None, 0, pos, freq, False)
        within(y, ref, size * HEAD_REL)
    a, b = q.head_norm_rope(qx, kx, i32(pos), dev(freq), dev(w), None)  # queries normed, keys not
    within(a, *[f(A.heads(host64(qx), w, 1e-6, pos, freq, False)) for f in (lambda r: r[0], lambda r: r[1] * HEAD_REL)])
    within(b, *[f(A.heads(host64(kx), None, 0, pos, freq, False)) for f in (lambda r: r[0], lambda r: r[1] * HEAD_REL)])
    a, b = q.head_norm_rope(qx, kx, None, None)  # neither: a copy
    assert torch.equal(a, qx) and torch.equal(b, kx)


def test_heads_of_zeros_and_extremes():
    x = torch.zeros((4, 2, 128), device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 0, 5] = float("inf")
    x[3, 1, 5] = float("nan")
    w = torch.ones(128, device="cuda")
    for eps in (1e-6, 0.0):
        y, _ = q.head_norm_rope(x, x, None, None, w, w, eps=eps)
        assert bool(torch.isnan(y[3, 0, 5])) and bool(torch.isnan(y[3, 1]).all())
        assert bool((y[2] - 1).abs().max() < 1e-6)
        if eps:
            assert bool((y[0] == 0).all()) and bool((y[1] - 1e-17).abs().max() < 1e-23)
        else:
            assert bool(torch.isnan(y[0]).all())
    assert q.head_norm_rope(x[:0], x[:0], None, None, w, w)[0].shape == (0, 2, 128)


# ---- the cache ---------------------------------------------------------------------------------

CACHES = ["f16", "bf16", "e4m3"]


def blank(pages, page, H, D, kind):
    c = q.KVCache.empty(pages, page, H, D, kind if kind == "e4m3" else DTYPES[kind])
    for t in (c.k, c.v, c.k_scales, c.v_scales):  # what pages hold before: NaN
        if t is not None:
            t.fill_(0x7F) if t.dtype == torch.uint8 else t.fill_(float("nan"))
    return c


def stored64(c, x):
    """The cache's values [pages, H, page, D]."""
    t = getattr(c, x)
    if c.k_scales is None:
        return host64(t)
    return A.values(to_host(t), to_host(getattr(c, x + "_scales")))


WRITES = [(1, 1, 16, 16), (5, 3, 80, 16), (33, 8, 128, 64), (70, 2, 256, 32), (129, 4, 64, 128), (7, 5, 112, 16), (2000, 1, 32, 256)]


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("x", sorted(DTYPES))
@pytest.mark.parametrize("T,H,D,page", WRITES)
def test_write_and_read(T, H, D, page, x, kind):
    g = np.random.default_rng([73, T, D])
    pages = -(-T // page) + 3
    c = blank(pages, page, H, D, kind)
    _, k, v = head_inputs(g, T, 1, H, D, DTYPES[x], T % 2 == 0)
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    left_out = g.random(T) < 0.1
    left_out[0] = False
    given = np.where(left_out, g.choice([-1, -(1 << 31), pages * page, (1 << 31) - 1], T), slots)
    before = [t.clone() for t in (c.k, c.v)]
    c.write(k, v, i32(given))
    at, row = slots[~left_out] // page, slots[~left_out] % page
    for name, src, old in (("k", k, before[0]), ("v", v, before[1])):
        t = getattr(c, name)
        if kind == "e4m3":
            codes, scales = A.quantize(host64(src)[~left_out])
            assert np.array_equal(to_host(t)[at, :, row], codes), name
            assert np.array_equal(to_host(getattr(c, name + "_scales"))[at, :, row], scales), name
        else:
            assert np.array_equal(host64(t)[at, :, row], host64(src.to(t.dtype))[~left_out]), name
        held = np.ones((pages, page), bool)
        held[at, row] = False
        same = to_host(t.view(torch.uint8)).reshape(pages, H, page, -1).transpose(0, 2, 1, 3)[held]
        assert np.array_equal(same, to_host(old.view(torch.uint8)).reshape(pages, H, page, -1).transpose(0, 2, 1, 3)[held])


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("out", sorted(DTYPES))
@pytest.mark.parametrize("H,D,page,lengths", [(1, 16, 16, [1]), (3, 80, 16, [17, 0, 333, 16, 1]), (8, 128, 64, [64, 65, 63, 0, 0, 700]),
                                              (5, 256, 32, [40] * 70), (2, 64, 128, [1] * 200 + [0] * 40 + [3])])
def test_read_packed_sequences(H, D, page, lengths, out, kind):
    g = np.random.default_rng([74, D, len(lengths)])
    B, need = len(lengths), [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    c = blank(pages, page, H, D, kind)
    order = g.permutation(pages)[:sum(need)].astype(np.int32)
    table = np.full((B, max(need) + 1), -7, np.int32)
    ends = np.cumsum(need)
    for b in range(B):
        table[b, :need[b]] = order[ends[b] - need[b]:ends[b]]
    T = sum(lengths)
    starts = np.concatenate([[0], np.cumsum(lengths)]) + 2  # two rows before the first sequence, three behind the last
    owner, t = np.repeat(np.arange(B), lengths), np.concatenate([np.arange(n) for n in lengths])
    slots = table[owner, t // page] * page + t % page
    _, k, v = head_inputs(g, T, 1, H, D, torch.float32, False)
    c.write(k, v, i32(slots))
    into = tuple(torch.full((T + 5, H, D), 7.0, device="cuda", dtype=DTYPES[out]) for _ in "kv")
    got = c.read(i32(table.flatten()).view(B, -1), i32(starts), T + 5, out=into)
    for name, y in zip("kv", got):
        assert bool((y[:2] == 7).all()) and bool((y[T + 2:] == 7).all())
        want = stored64(c, name)[table[owner, t // page], :, t % page]
        within(y[2:T + 2], want, np.abs(want) * 2.0 ** -24)
    with_new = c.read(i32(table.flatten()).view(B, -1), i32(starts - 2), T, dtype=DTYPES[out])
    assert all(torch.equal(a, b[2:T + 2]) for a, b in zip(with_new, got))


def test_pages_that_are_none():
    for kind in CACHES:
        c = blank(4, 16, 2, 32, kind)
        k = torch.ones((40, 2, 32), device="cuda")
        c.write(k, k, i32(range(40)))
        table = torch.tensor([[0, 9, 2], [0, 1, -1], [0, 1, 2]], dtype=torch.int32, device="cuda")
        out = c.read(table, i32([0, 40, 80, 160]), 160, dtype=torch.float32)
        for y in out:
            nan = torch.isnan(y).flatten(1)
            assert not bool(nan[:16].any()) and bool(nan[16:32].all()) and not bool(nan[32:72].any()) and bool(nan[72:80].all())
            assert not bool(nan[80:120].any()) and bool(nan[128:].all())  # past the table's three columns
        if kind == "e4m3":
            continue
        y = c.attend(torch.ones((3, 2, 32), device="cuda", dtype=c.dtype), table, i32([40, 30, 40]))
        assert bool(torch.isnan(y[0]).all()) and not bool(torch.isnan(y[1:]).any())


def test_write_infinities_and_ties():
    c = blank(1, 16, 1, 32, "e4m3")
    x = torch.zeros((6, 1, 32), device="cuda")
    x[0, 0, 3] = float("inf")
    x[1, 0, 3] = float("nan")
    x[2] = torch.arange(32, device="cuda") / 64 + 7.0 / 16  # many quotients on the middle of two codes
    x[3, 0, 0] = -0.0
    x[4, 0, :2] = torch.tensor([3e38, 1e-30], device="cuda")
    x[5] = 1e-40
    c.write(x, x, i32(range(6)))
    codes, scales = A.quantize(host64(x))
    assert np.array_equal(to_host(c.k_scales)[0, 0, :6], scales[:, 0], equal_nan=True)
    assert np.array_equal(to_host(c.k)[0, 0, 2:6], codes[2:, 0])


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("x", sorted(DTYPES))
@pytest.mark.parametrize("T,Hq,H,D,R", HEADS)
def test_norm_rope_write_is_the_two_calls(T, Hq, H, D, R, x, kind):
    g = np.random.default_rng([75, T, D])
    page = 16
    pages = -(-T // page) + 1
    qx, kx, vx = head_inputs(g, T, Hq, H, D, DTYPES[x], T % 2 == 1)
    w, pos, freq = dev(1 + g.random(D)), i32(g.integers(0, 1 << 20, T)), dev(frequencies(R))
    slots = g.permutation(pages * page)[:T]
    slots[T // 3] = -1
    for interleaved in (False, True):
        for t in ([DTYPES[kind]] if kind != "e4m3" else list(DTYPES.values())):
            one, two = blank(pages, page, H, D, kind), blank(pages, page, H, D, kind)
            got = one.norm_rope_write(qx, kx, vx, i32(slots), pos, freq, w, w, eps=EPS, interleaved=interleaved, dtype=t)
            q2, k2 = q.head_norm_rope(qx, kx, pos, freq, w, w, eps=EPS, interleaved=interleaved, dtype=t)
            two.write(k2, k2, i32(slots))
            v_only = blank(pages, page, H, D, kind)
            v_only.write(vx, vx, i32(slots))
            assert torch.equal(got, q2)
            for a, b in ((one.k, two.k), (one.v, v_only.v), (one.k_scales, two.k_scales), (one.v_scales, v_only.v_scales)):
                if a is not None:
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- attention over the cache ------------------------------------------------------------------

def score_error(reach, D):
    """Error of a probability relative to it: a score's products are exact and their sum rounds at most D times (2^-24 of
    the sum of magnitudes), the scale twice; exp2 and its argument's rounding; then the same once more for the sum of all."""
    return 2 * (reach * ((D + 4) * 2.0 ** -24) + 4 * 2.0 ** -23)


def rounding_noise(spread, noise, step):
    """Error of a sum whose terms are rounded to half steps of `step`: independent, so six times their root mean square
    (step / sqrt 3 each), and at most all of them."""
    return step * np.minimum(spread, 6 / np.sqrt(3) * noise)


def filled(g, lengths, page, H, D, kind, channels=4.0):
    """A cache that holds sequences of these lengths on shuffled pages (NaN elsewhere), its table, keys and values."""
    B, need = len(lengths), [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    c = blank(pages, page, H, D, kind)
    order = g.permutation(pages)[:sum(need)]
    table = np.full((B, max(max(need), 1)), -1, np.int32)
    ends = np.cumsum(need)
    for b in range(B):
        table[b, :need[b]] = order[ends[b] - need[b]:ends[b]]
    owner, t = np.repeat(np.arange(B), lengths), np.concatenate([np.arange(n) for n in lengths]).astype(np.int64)
    T = len(t)
    k = g.standard_normal((T, H, D))
    k[..., ::16] *= channels
    if T:
        c.write(dev(k), dev(g.standard_normal((T, H, D))), i32(table[owner, t // page] * page + t % page))
    return c, table, owner, t


def attend_reference(c, table, lengths, qx, scale):
    """Outputs and bound of the oracle for every sequence and head."""
    page, H = c.page, c.heads
    B, Hq, D = qx.shape
    parts = np.zeros((3, B, Hq, D))
    reach = np.zeros((B, Hq, 1))
    kv = [stored64(c, x) for x in "kv"]
    for b, n in enumerate(lengths):
        t = np.arange(n)
        rows = [a[table[b, t // page], :, t % page] for a in kv]
        for h in range(Hq):
            g = h * H // Hq
            o = A.attend(host64(qx[b, h])[None], rows[0][:, g], rows[1][:, g], scale, np.ones((1, n), bool))
            for i in range(3):
                parts[i, b, h] = o[i][0]
            reach[b, h] = o[3][0]
    out, spread, noise = parts
    # P as two 16-bit numbers: 2^-17 of a term and less; sums over the keys in fp32, in chains of at most a few hundred adds
    bound = spread * (score_error(reach, D) + 2.0 ** -16 + 512 * 2.0 ** -24)
    return out, bound


ATTEND = [  # B lengths, page, Hq, H, D
    ([1], 16, 1, 1, 16), ([0], 16, 2, 2, 32), ([777], 64, 16, 8, 128), ([5, 0, 31, 32, 33, 127, 128, 129, 500], 16, 8, 4, 128),
    ([300, 17, 64], 32, 21, 3, 80), ([1, 2, 15, 16, 17], 128, 6, 1, 256), ([2000, 1999], 256, 40, 2, 64),
    ([100] * 40, 16, 4, 4, 112), ([4097], 64, 17, 1, 96), ([3000, 10], 16, 33, 1, 128), ([600], 16, 7, 7, 144),
    ([300, 257, 1, 0] + [40] * 60, 16, 10, 5, 64), ([400] + [33] * 36, 32, 8, 8, 128), ([2300, 2049, 0] + [20] * 30, 16, 4, 4, 96),
    ([300] + [16] * 140, 16, 2, 2, 160), ([290] + [20] * 140, 16, 2, 2, 256), ([400] + [33] * 36, 32, 8, 8, 192),
    ([300, 20], 16, 4, 2, 32), ([700, 90], 64, 3, 1, 176),
]


@pytest.mark.parametrize("t", sorted(HALF))
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("lengths,page,Hq,H,D", ATTEND)
def test_attend(lengths, page, Hq, H, D, codes, t):
    g = np.random.default_rng([76, len(lengths), Hq, D])
    c, table, _, _ = filled(g, lengths, page, H, D, "e4m3" if codes else t)
    B = len(lengths)
    wide = dev(g.standard_normal((B, Hq, D + 8)) * 1.5, HALF[t])
    qx = wide[:, :, 4:4 + D]  # a slice: strided rows
    tab = i32(table.flatten()).view(B, -1)
    ref, bound = attend_reference(c, table, lengths, qx, D ** -0.5)
    got = c.attend(qx, tab, i32(lengths))
    within(got, ref, bound, "default")
    within(c.attend(qx, tab, i32(lengths), max_length=max(lengths)), ref, bound, "longest known")
    within(c.attend(qx, tab, i32(lengths), max_length=0), ref, bound, "one piece")
    assert torch.equal(got, c.attend(qx.contiguous(), tab, i32(lengths)))
    wide_table = torch.cat([tab, torch.full((B, 5000 // page), -1, dtype=torch.int32, device="cuda")], 1)
    within(c.attend(qx, wide_table, i32(lengths)), ref, bound, "wide table")
    ref, bound = attend_reference(c, table, lengths, qx, 0.7)
    out = torch.full((B, Hq, D), 9.0, device="cuda", dtype=HALF[t])
    assert c.attend(qx, tab, i32(lengths), scale=0.7, out=out) is out
    within(out, ref, bound, "scale")


def test_attend_lengths_past_the_table_and_below_zero():
    g = np.random.default_rng(77)
    c, table, _, _ = filled(g, [64, 64, 64], 16, 2, 64, "bf16")
    qx = dev(g.standard_normal((3, 4, 64)), torch.bfloat16)
    tab = i32(table.flatten()).view(3, -1)
    full = c.attend(qx, tab, i32([64, 64, 0]))
    assert torch.equal(full, c.attend(qx, tab, i32([100, 2 ** 31 - 1, -5])))
    assert bool((full[2] == 0).all())
    none = c.attend(qx, torch.empty((3, 0), dtype=torch.int32, device="cuda"), i32([5, 0, 1]))
    assert bool((none == 0).all())
    assert c.attend(qx[:0], tab[:0], i32([])).shape == (0, 4, 64)


def test_attend_infinities():
    """Past a sequence's end anything may lie; NaN and Inf inside reach the rows that see them and no others."""
    g = np.random.default_rng(78)
    for kind in CACHES:
        c, table, _, _ = filled(g, [70, 70], 16, 2, 64, kind)
        tab, n = i32(table.flatten()).view(2, -1), i32([70, 70])
        qx = dev(g.standard_normal((2, 4, 64)), c.dtype if kind != "e4m3" else torch.float16)
        want = c.attend(qx, tab, n)
        assert bool(torch.isfinite(want).all())
        bad = torch.zeros((1, 2, 64), device="cuda")
        bad[:, 1, 5] = float("nan")
        c.write(bad, bad, i32([int(table[0, 4]) * 16 + 5]))  # token 69 of the first
        got = c.attend(qx, tab, n)
        assert bool(torch.isnan(got[0, 2:]).any(1).all()) and torch.equal(got[1], want[1])
        assert bool(torch.isfinite(got[0, :2]).all())
        assert torch.equal(c.attend(qx, tab, i32([69, 70]))[1], want[1])
        assert bool(torch.isfinite(c.attend(qx, tab, i32([69, 70]))).all())  # it lies past the end now
    qx = torch.full((1, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    c, table, _, _ = filled(g, [40], 16, 2, 64, "bf16")
    assert bool(torch.isnan(c.attend(qx, i32(table.flatten()).view(1, -1), i32([40]))).all())


def test_attend_sharp_and_flat():
    """One token far above all others; all scores equal; scores that rise to the end (every tile moves the maximum)."""
    g = np.random.default_rng(79)
    H, D, n, page = 1, 64, 3001, 16
    for t in HALF.values():
        kind = "f16" if t == torch.float16 else "bf16"
        c, table, _, tok = filled(g, [n], page, H, D, kind)
        k = np.zeros((n, H, D))
        k[:, 0, 0] = np.linspace(-200, 200, n)
        v = g.standard_normal((n, H, D))
        c.write(dev(k), dev(v), i32(table[0, tok // page] * page + tok % page))
        tab = i32(table.flatten()).view(1, -1)
        qx = torch.zeros((1, 4, D), device="cuda", dtype=t)
        qx[0, 1, 0], qx[0, 2, 0], qx[0, 3, 0] = 8.0, -8.0, 100.0
        ref, bound = attend_reference(c, table, [n], qx, 0.125)
        within(c.attend(qx, tab, i32([n])), ref, bound)
        within(c.attend(qx, tab, i32([n]), max_length=1), ref, bound)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_cache_beyond_4_gib(kind):
    """Pages whose bytes lie past 2^32: written, read back and attended to."""
    g = np.random.default_rng(80)
    H, D, page = 8, 128, 256
    pages = (int(4.6 * 2 ** 30) if kind == "e4m3" else int(5 * 2 ** 30)) // (H * D * page * (1 if kind == "e4m3" else 2))
    c = q.KVCache.empty(pages, page, H, D, "e4m3" if kind == "e4m3" else torch.bfloat16)
    n = 3 * page - 5
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    t = np.arange(n)
    slots = i32(table[0, t // page] * page + t % page)
    k, v = (dev(g.standard_normal((n, H, D))) for _ in "kv")
    c.write(k, v, slots)
    tab = i32(table.flatten()).view(1, -1)
    rk, rv = c.read(tab, i32([0, n]), n, dtype=torch.float32)
    for got, src in ((rk, k), (rv, v)):
        err = HALF_STEP[torch.bfloat16] if kind == "bf16" else 2.0 ** -4
        assert bool(((got - src).abs() <= src.abs() * err + src.abs().amax(-1, keepdim=True) * 2.0 ** -17).all())
    qx = dev(g.standard_normal((1, 16, D)), torch.bfloat16)
    small = q.KVCache.empty(3, page, H, D, "e4m3" if kind == "e4m3" else torch.bfloat16)
    small.write(k, v, i32(range(n)))
    want = small.attend(qx, i32([0, 1, 2]).view(1, 3), i32([n]))
    assert torch.equal(c.attend(qx, tab, i32([n])), want)


# ---- prompts -----------------------------------------------------------------------------------

def prompt_inputs(g, ns, ms, Hq, H, D, dtype, fused):
    T, Tk = sum(ns), sum(ms)
    if fused:
        rows = g.standard_normal((T, Hq + 2 * H, D))
        rows[:, :Hq] *= 1.5
        rows[:, Hq:Hq + H, ::16] *= 4
        rows = dev(rows, dtype)
        return rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
    k = g.standard_normal((Tk, H, D))
    k[..., ::16] *= 4
    return dev(g.standard_normal((T, Hq, D)) * 1.5, dtype), dev(k, dtype), dev(g.standard_normal((Tk, H, D)), dtype)


def starts(ns):
    return i32(np.concatenate([[0], np.cumsum(ns)]))


def prompt_reference(qx, k, v, ns, ms, scale, causal, step):
    Hq, H, D = qx.shape[1], k.shape[1], qx.shape[2]
    q64, k64, v64 = host64(qx), host64(k), host64(v)
    out, bound = np.zeros(q64.shape), np.zeros(q64.shape)
    a = b = 0
    for n, m in zip(ns, ms):
        seen = A.causal(n, m) if causal else np.ones((n, m), bool)
        for h in range(Hq):
            g = h * H // Hq
            o, spread, noise, reach = A.attend(q64[a:a + n, h], k64[b:b + m, g], v64[b:b + m, g], scale, seen)
            out[a:a + n, h] = o
            bound[a:a + n, h] = spread * (score_error(reach, D) + (m + 16) * 2.0 ** -24) + rounding_noise(spread, noise, step)
        a, b = a + n, b + m
    return out, bound


PROMPTS = [  # queries, keys, Hq, H, D
    ([1], [1], 1, 1, 16), ([7], [7], 4, 2, 128), ([128], [128], 2, 2, 128), ([130, 1, 0, 64, 63, 65, 33], None, 4, 2, 64),
    ([200], [260], 6, 2, 80), ([5, 40], [300, 41], 3, 1, 256), ([9], [4], 2, 1, 32), ([150, 30], [100, 0], 2, 1, 64),
    ([0, 0, 3], [5, 0, 3], 2, 2, 96), ([1] * 70 + [2, 129], None, 1, 1, 48), ([321], [321], 2, 1, 112), ([64, 64], [64, 128], 16, 8, 128),
    ([265], [300], 63, 21, 64), ([260, 5], [270, 260], 64, 4, 128), ([540], [1030], 61, 61, 32), ([300], [301], 222, 2, 32),
    ([150, 160], [250, 160], 224, 8, 128), ([1, 513], None, 6, 6, 80),
    ([70, 9], [90, 9], 2, 1, 160), ([40, 130], None, 3, 3, 192), ([129], [140], 8, 2, 224), ([300], [300], 4, 2, 32),
]


@pytest.mark.parametrize("t", sorted(HALF))
@pytest.mark.parametrize("ns,ms,Hq,H,D", PROMPTS)
def test_prompt(ns, ms, Hq, H, D, t):
    g = np.random.default_rng([81, len(ns), sum(ns), D])
    same = ms is None or ms == ns
    ms = ns if ms is None else ms
    qx, k, v = prompt_inputs(g, ns, ms, Hq, H, D, HALF[t], same)
    qs, ks = starts(ns), None if same else starts(ms)
    for causal in (True, False):
        ref, bound = prompt_reference(qx, k, v, ns, ms, D ** -0.5, causal, HALF_STEP[HALF[t]])
        got = q.attend_prompt(qx, k, v, qs, ks, causal=causal)
        within(got, ref, bound, f"causal {causal}")
        assert torch.equal(got, q.attend_prompt(qx.contiguous(), k.contiguous(), v.contiguous(), qs, ks, causal=causal))
    ref, bound = prompt_reference(qx, k, v, ns, ms, 0.3, True, HALF_STEP[HALF[t]])
    out = torch.full_like(qx, 9.0, memory_format=torch.contiguous_format)
    assert q.attend_prompt(qx, k, v, qs, ks, scale=0.3, out=out) is out
    within(out, ref, bound, "scale")


@pytest.mark.parametrize("B", [63, 64, 65, 4097, 5000])
def test_many_short_sequences(B):
    """More sequences than lanes, many of them empty: the tiles' search for theirs, and that of packed rows for theirs."""
    g = np.random.default_rng([90, B])
    H, D, page = 1, 16, 16
    ns = g.choice([0, 1, 2, 5], B)
    ns[B // 2], ns[-1] = 300, 130
    before = g.choice([0, 3], B)
    ms = ns + before
    T, Tk = int(ns.sum()), int(ms.sum())
    qx, k, v = prompt_inputs(g, ns, ms, 2, H, D, torch.bfloat16, False)
    got = host64(q.attend_prompt(qx, k, v, starts(ns), starts(ms)))
    ends, kends = np.cumsum(ns), np.cumsum(ms)
    seen = np.zeros((T, Tk), bool)  # a block of keys for every row
    for b in range(B):
        seen[ends[b] - ns[b]:ends[b], kends[b] - ms[b]:kends[b]] = A.causal(ns[b], ms[b])
    for h in range(2):
        o, spread, noise, reach = A.attend(host64(qx[:, h]), host64(k[:, 0]), host64(v[:, 0]), D ** -0.5, seen)
        bound = spread * (score_error(reach, D) + 400 * 2.0 ** -24) + rounding_noise(spread, noise, HALF_STEP[torch.bfloat16])
        tol = bound + (np.abs(o) + bound) * HALF_STEP[torch.bfloat16] + SMALLEST[torch.bfloat16]
        assert np.all(np.abs(got[:, h] - o) <= tol)
    need = -(-ms // page)
    table = np.full((B, int(need.max())), -1, np.int32)
    order = g.permutation(int(need.sum()))
    at = np.cumsum(need) - need
    for b in range(B):
        table[b, :need[b]] = order[at[b]:at[b] + need[b]]
    c = blank(int(need.sum()), page, H, D, "bf16")
    owner, t = np.repeat(np.arange(B), ms), np.concatenate([np.arange(n) for n in ms])
    c.write(k, v, i32(table[owner, t // page] * page + t % page))
    rk, rv = c.read(i32(table.flatten()).view(B, -1), starts(ms), Tk)
    assert torch.equal(rk, k) and torch.equal(rv, v)


@pytest.mark.parametrize("n,Hq,D", [(70, 2, 128), (300, 4, 96), (65, 2, 256), (40, 1, 32)])
def test_prompt_queries_and_outputs_at_any_element(n, Hq, D):
    g = np.random.default_rng([98, D])
    qx, k, v = prompt_inputs(g, [n], [n], Hq, 1, D, torch.bfloat16, False)
    want = q.attend_prompt(qx, k, v, starts([n]))
    rows = torch.full((n, Hq * D + 3), float("nan"), device="cuda", dtype=torch.bfloat16)
    odd = rows[:, 1:1 + Hq * D].unflatten(1, (Hq, D))
    odd.copy_(qx)
    room = torch.full((n * Hq * D + 2,), 9.0, device="cuda", dtype=torch.bfloat16)
    out = room[1:-1].view(n, Hq, D)
    q.attend_prompt(odd, k, v, starts([n]), out=out)
    assert torch.equal(out, want) and room[0] == 9 and room[-1] == 9


def test_prompt_rows_of_no_sequence():
    g = np.random.default_rng(82)
    qx, k, v = prompt_inputs(g, [100], [100], 2, 1, 64, torch.bfloat16, True)
    out = torch.full((100, 2, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    q.attend_prompt(qx, k, v, i32([3, 20, 90]), out=out)
    assert bool((out[:3] == 9).all()) and bool((out[90:] == 9).all())
    want = q.attend_prompt(qx[3:90], k[3:90], v[3:90], i32([0, 17, 87]))
    assert torch.equal(out[3:90], want)
    q.attend_prompt(qx, k, v, i32([0, 0, 0]), out=out)  # sequences without queries: nothing is written
    assert torch.equal(out[3:90], want) and bool((out[90:] == 9).all())
    bad = q.attend_prompt(qx, k, v, i32([-5, 50, 1000]))  # kept within the tensors
    assert bool(torch.isfinite(bad).all())
    assert q.attend_prompt(qx[:0], k[:0], v[:0], i32([0])).shape == (0, 2, 64)
    assert q.attend_prompt(qx[:0], k[:0], v[:0], i32([0, 0])).shape == (0, 2, 64)
    empty = q.attend_prompt(qx, k[:0], v[:0], i32([0, 100]), i32([0, 0]))  # queries without keys
    assert bool((empty == 0).all())


@pytest.mark.parametrize("D", [48, 128, 256])
@pytest.mark.parametrize("t", sorted(HALF))
def test_prompt_infinities_in_masked_places(D, t):
    """Keys and values that a row does not see, NaN and infinite ones among them, leave its output as it was."""
    g = np.random.default_rng([83, D])
    n, at = 300, 205
    qx, k, v = prompt_inputs(g, [n], [n], 2, 1, D, HALF[t], False)
    s = starts([n])
    want = q.attend_prompt(qx, k, v, s)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for where in "kv":
            k2, v2 = k.clone(), v.clone()
            (k2 if where == "k" else v2)[at, 0, D // 2] = bad
            got = q.attend_prompt(qx, k2, v2, s)
            ref, bound = prompt_reference(qx[:at], k[:at], v[:at], [at], [at], D ** -0.5, True, HALF_STEP[HALF[t]])
            within(got[:at], ref, bound, f"{where} {bad}")
            if where == "v":
                assert not bool(torch.isfinite(got[at:, :, D // 2]).any())
                others = torch.arange(D, device="cuda") != D // 2
                assert bool(torch.isfinite(got[at:][..., others]).all())
            elif bad != bad:
                assert bool(torch.isnan(got[at:]).all())
    # the lowest values (bf16: as low as fp32 holds the scores of): scores far from zero, equal for a row
    low = torch.full_like(k, torch.finfo(HALF[t]).min / (512 if t == "bf16" else 1))
    y = q.attend_prompt(torch.ones_like(qx), low, v, s)
    mean = v.double().cumsum(0) / torch.arange(1, n + 1, device="cuda").view(-1, 1, 1)
    assert bool(((y.double() - mean).abs() <= 2 * HALF_STEP[HALF[t]] * 4 + 1e-3).all())
    del want


@pytest.mark.parametrize("t", sorted(HALF))
@pytest.mark.parametrize("ns,ms,Hq,H,D", [([260, 70, 1], [400, 500, 90], 8, 2, 128), ([150], [150], 3, 3, 64), ([200, 65], [200, 70], 4, 2, 256),
                                          ([130], [100], 2, 2, 48), ([265], [300], 64, 4, 128), ([300], [301], 224, 2, 64),
                                          ([100], [130], 4, 2, 176), ([140, 70], None, 2, 1, 96), ([300], [300], 2, 2, 32)])
def test_prompt_infinities_among_many_values(ns, ms, Hq, H, D, t):
    """NaN and infinite values in a tenth of the rows: what a row sees of a column decides, tile by tile."""
    g = np.random.default_rng([96, D])
    ms = ns if ms is None else ms
    qx, k, v = prompt_inputs(g, ns, ms, Hq, H, D, HALF[t], False)
    Tk = sum(ms)
    bad = np.zeros((Tk, H, D), bool)
    rows = g.random(Tk) < 0.1
    bad[rows] = g.random((int(rows.sum()), H, D)) < 0.02
    spoiled = np.where(bad, g.choice([np.nan, np.inf, -np.inf], bad.shape), host64(v))
    ref, bound = prompt_reference(qx, k, dev(np.where(bad, 0, host64(v)), HALF[t]), ns, ms, D ** -0.5, True, HALF_STEP[HALF[t]])
    got = host64(q.attend_prompt(qx, k, dev(spoiled, HALF[t]), starts(ns), starts(ms)))
    a = b = 0
    met = np.zeros(ref.shape, bool)
    for n, m in zip(ns, ms):
        seen = A.causal(n, m)
        for h in range(Hq):
            met[a:a + n, h] = seen.astype(int) @ bad[b:b + m, h * H // Hq].astype(int) > 0
        a, b = a + n, b + m
    assert met.any() and not met.all()
    assert not np.isfinite(got[met]).any()
    tol = bound + (np.abs(ref) + bound) * HALF_STEP[HALF[t]] + SMALLEST[HALF[t]]
    assert np.all(np.abs(got - ref)[~met] <= tol[~met])


def test_read_past_many_empty_sequences():
    """Rows of one workgroup on both sides of thousands of empty sequences."""
    g = np.random.default_rng(97)
    ns = np.zeros(9000, int)
    ns[[0, 1, 4000, 4001, 8999]] = 3, 2, 1, 4, 5
    c = blank(5, 16, 2, 32, "bf16")
    k, v = (dev(g.standard_normal((15, 2, 32)), torch.bfloat16) for _ in "kv")
    owner, t = np.repeat(np.arange(9000), ns), np.concatenate([np.arange(n) for n in ns])
    table = np.full((9000, 1), -1, np.int32)
    table[ns > 0, 0] = g.permutation(5)
    c.write(k, v, i32(table[owner, 0] * 16 + t))
    rk, rv = c.read(i32(table.flatten()).view(-1, 1), starts(ns), 15)
    assert torch.equal(rk, k) and torch.equal(rv, v)


def test_prompt_sharp_and_flat():
    g = np.random.default_rng(84)
    n, D = 700, 64
    for t in HALF.values():
        k = np.zeros((n, 1, D))
        k[:, 0, 0] = np.linspace(-200, 200, n)
        qx = np.zeros((n, 4, D))
        qx[:, 1, 0], qx[:, 2, 0], qx[:, 3, 0] = 8.0, -8.0, 100.0
        qx, k, v = dev(qx, t), dev(k, t), dev(g.standard_normal((n, 1, D)), t)
        ref, bound = prompt_reference(qx, k, v, [n], [n], 0.125, True, HALF_STEP[t])
        within(q.attend_prompt(qx, k, v, starts([n]), scale=0.125), ref, bound)


def test_rows_beyond_4_gib():
    """Rows of wide buffers whose offsets pass 2^32 bytes."""
    g = np.random.default_rng(85)
    T, H, D = 5000, 2, 64
    wide = torch.empty((T, 1 << 19), dtype=torch.bfloat16, device="cuda")
    rows = wide[:, :4 * H * D].unflatten(1, (4 * H, D))
    rows.copy_(torch.randn((T, 4 * H, D), device="cuda"))
    qx, k, v = rows[:, :2 * H], rows[:, 2 * H:3 * H], rows[:, 3 * H:]
    s = i32([0, T - 300, T])
    assert torch.equal(q.attend_prompt(qx, k, v, s), q.attend_prompt(qx.contiguous(), k.contiguous(), v.contiguous(), s))
    pos, freq = i32(g.integers(0, 9999, T)), dev(frequencies(D))
    a, b = q.head_norm_rope(qx, k, pos, freq), q.head_norm_rope(qx.contiguous(), k.contiguous(), pos, freq)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = [q.KVCache.empty(320, 16, H, D) for _ in range(2)]
    c[0].write(k, v, i32(range(T)))
    c[1].write(k.contiguous(), v.contiguous(), i32(range(T)))
    assert torch.equal(c[0].k, c[1].k) and torch.equal(c[0].v, c[1].v)


# ---- together ----------------------------------------------------------------------------------

class Layer:
    """Projections, norms, cache and attention of a decoder layer's first half."""

    def __init__(self, g, width, Hq, H, D):
        self.Hq, self.H, self.D = Hq, H, D
        sizes = {"q": (Hq * D, width), "k": (H * D, width), "v": (H * D, width), "o": (width, Hq * D)}
        self.m = {n: q.QMatrix(q.quantize(dev(g.standard_normal((M, K)) * K ** -0.5), "q8_0"), "q8_0", M, K)
                  for n, (M, K) in sizes.items()}
        self.qw, self.kw = (dev(1 + 0.1 * g.standard_normal(D)) for _ in "qk")
        self.freq = dev(frequencies(D))

    def heads(self, x):
        return (self.m[n].gemm(x).view(x.shape[0], -1, self.D) for n in "qkv")


@pytest.mark.parametrize("kind", CACHES)
def test_prompt_in_parts_then_decode(kind):
    """Projections, norms and rotation, cache, attention, output projection: two prompts that arrive in two parts, then
    tokens one by one, against the whole sequences in one go."""
    g = np.random.default_rng(86)
    width, Hq, H, D, page = 256, 8, 2, 64, 16
    layer = Layer(g, width, Hq, H, D)
    t = torch.bfloat16 if kind == "bf16" else torch.float16
    lengths, first, new = [75, 40], [50, 11], 4
    xs = [dev(g.standard_normal((n + new, width)), torch.float16) for n in lengths]
    cache = q.KVCache.empty(16, page, H, D, kind if kind == "e4m3" else t)
    table = np.array([[3, 0, 7, 9, 1, -1], [12, 5, 2, -1, -1, -1]], np.int32)
    tab = i32(table.flatten()).view(2, -1)

    def slots(b, lo, hi):
        return [int(table[b, i // page]) * page + i % page for i in range(lo, hi)]

    def part(lo, hi):
        x = torch.cat([x[a:b] for x, a, b in zip(xs, lo, hi)])
        qx, kx, vx = layer.heads(x)
        pos = [i for a, b in zip(lo, hi) for i in range(a, b)]
        at = [s for i, (a, b) in enumerate(zip(lo, hi)) for s in slots(i, a, b)]
        return cache.norm_rope_write(qx, kx, vx, i32(at), i32(pos), layer.freq, layer.qw, layer.kw, dtype=t)

    outs = [[], []]

    def keep(y, lo, hi):
        at = 0
        for i, (a, b) in enumerate(zip(lo, hi)):
            outs[i].append(y[at:at + b - a])
            at += b - a

    for lo, hi in (([0, 0], first), (first, lengths)):
        qr = part(lo, hi)
        k, v = cache.read(tab, starts(hi), sum(hi), dtype=t)
        y = q.attend_prompt(qr, k, v, starts([b - a for a, b in zip(lo, hi)]), starts(hi))
        keep(y, lo, hi)
    for i in range(new):
        lo = [n + i for n in lengths]
        hi = [n + 1 for n in lo]
        keep(cache.attend(part(lo, hi), tab, i32(hi)), lo, hi)

    # the whole sequences: fp64 attention over what the cache holds, for the queries the calls made
    for b, n in enumerate(lengths):
        n += new
        got = torch.cat(outs[b])
        qx, kx, _ = layer.heads(xs[b])
        qr = q.head_norm_rope(qx, kx, i32(range(n)), layer.freq, layer.qw, layer.kw, dtype=t)[0]
        tok = np.arange(n)
        k64, v64 = (stored64(cache, x)[table[b, tok // page], :, tok % page] for x in "kv")
        for h in range(Hq):
            o, spread, noise, reach = A.attend(host64(qr[:, h]), k64[:, h * H // Hq], v64[:, h * H // Hq], D ** -0.5,
                                               A.causal(n, n))
            step = HALF_STEP[t]
            # a projection's fp32 sums round differently by its number of tokens, so that a query may move by a step (two
            # halves); what the cache gives back is rounded once more: a score moves by three half steps of the sum of
            # magnitudes, a probability by twice that; a value and a probability are rounded once each
            moved = 3 * step * reach
            within(got[:, h], o, spread * (score_error(reach, D) + 2 * moved + 2 * step + n * 2.0 ** -24), f"{kind} {b} {h}")
        y = layer.m["o"].gemm(got.flatten(1).to(torch.float16))
        assert y.shape == (n, width) and bool(torch.isfinite(y).all())


def test_captured_step_replays():
    """A decode step in a graph: replayed with new inputs, lengths and tables in its buffers, eager work between."""
    g = np.random.default_rng(87)
    B, Hq, H, D, page = 3, 8, 2, 128, 16
    cache = q.KVCache.empty(64, page, H, D, "e4m3")
    w, freq = dev(1 + 0.1 * g.standard_normal(D)), dev(frequencies(D))
    tab = i32(g.permutation(64)[:60]).view(B, 20)
    qx, kx, vx = (dev(g.standard_normal((B, n, D)), torch.bfloat16) for n in (Hq, H, H))
    pos, lens, slots = i32([0] * B), i32([1] * B), i32([0] * B)
    cache.write(*(dev(g.standard_normal((64 * page, H, D))) for _ in "kv"), i32(range(64 * page)))

    def step():
        qr = cache.norm_rope_write(qx, kx, vx, slots, pos, freq, w, w)
        return cache.attend(qr, tab, lens, max_length=320)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        n = g.integers(1, 320, B)
        for t in (qx, kx, vx):
            t.copy_(dev(g.standard_normal(t.shape), torch.bfloat16))
        pos.copy_(i32(n - 1))
        lens.copy_(i32(n))
        slots.copy_(i32([int(tab[b, (n[b] - 1) // page]) * page + (n[b] - 1) % page for b in range(B)]))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step()), turn
        torch.cuda.synchronize()


def test_streams_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give alone."""
    g = np.random.default_rng(88)
    c, table, _, _ = filled(g, [5000, 3000], 64, 2, 128, "bf16")
    tab, n = i32(table.flatten()).view(2, -1), i32([5000, 3000])
    qs = [dev(g.standard_normal((2, 8, 128)), torch.bfloat16) for _ in range(2)]
    want = [c.attend(x, tab, n) for x in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(c.attend(qs[i], tab, n))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_cache_handles():
    c = q.KVCache.empty(2, 16, 1, 32, "e4m3")
    x = torch.randn((20, 1, 32), device="cuda")
    c.write(x, x, i32(range(20)))
    other, deep = copy.copy(c), copy.deepcopy(c)
    assert other.k is c.k and deep.k is not c.k and torch.equal(deep.k, c.k)
    c.close()
    c.close()
    with pytest.raises(q.QmmError, match="NULL"):
        c.write(x, x, i32(range(20)))
    for columns in (0, 32):
        with pytest.raises((q.QmmError, ValueError)):
            c.attend(torch.zeros((1, 1, columns), device="cuda", dtype=torch.bfloat16), i32([0]).view(1, 1), i32([1]))
    rows = torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2)
    want = deep.read(rows, i32([0, 20]), 20, dtype=torch.float32)
    del c
    assert all(torch.equal(a, b) for a, b in zip(other.read(rows, i32([0, 20]), 20, dtype=torch.float32), want))
    codes = q.KVCache(other.k.view(torch.float8_e4m3fn), other.v.view(torch.float8_e4m3fn), other.k_scales, other.v_scales)
    assert all(torch.equal(a, b) for a, b in zip(codes.read(rows, i32([0, 20]), 20, dtype=torch.float32), want))


def test_starts_that_decrease_stay_inside():
    """Not allowed, and harmless: rows of the tensors only, some of them written."""
    g = np.random.default_rng(91)
    T = 700
    qx, k, v = prompt_inputs(g, [T], [T], 4, 2, 64, torch.bfloat16, False)
    guard = torch.full((T + 64, 4, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    c = blank(50, 16, 2, 64, "bf16")
    c.write(k, v, i32(range(T)))
    rows = i32(range(44)).view(1, 44).expand(4, 44).contiguous()
    for s in ([0, 300, 100, 700, 650], [700, 0, 700, 0, 700], [0, -50, 2 ** 31 - 1, -(2 ** 31), 40], [500, 400, 300, 200, 100]):
        out = guard[32:T + 32]
        q.attend_prompt(qx, k, v, i32(s), out=out)
        assert bool((guard[:32] == 9).all()) and bool((guard[T + 32:] == 9).all())
        assert bool(torch.isfinite(guard).all())
        into = tuple(torch.full((T + 64, 2, 64), 9.0, device="cuda") for _ in "kv")
        c.read(rows, i32(s), T, out=tuple(t[32:T + 32] for t in into))
        assert all(bool((t[:32] == 9).all()) and bool((t[T + 32:] == 9).all()) for t in into)


def test_calls_through_ctypes_are_the_same(monkeypatch):
    """What the native calls decline is made in Python: with the same results."""
    from block_quantized_weight_matmul_amd import attention
    assert attention._calls is not None
    g = np.random.default_rng(92)
    c, table, _, _ = filled(g, [500, 300], 16, 2, 64, "e4m3")
    other, tab, n = copy.deepcopy(c), i32(table.flatten()).view(2, -1), i32([500, 300])
    qx, kx, vx = head_inputs(g, 2, 4, 2, 64, torch.bfloat16, True)
    pos, freq, w = i32([499, 299]), dev(frequencies(64)), dev(1 + g.random(64))
    slots = i32([int(table[0, 499 // 16]) * 16 + 499 % 16, int(table[1, 299 // 16]) * 16 + 299 % 16])
    ps, pk = starts([1, 1]), starts([500, 300])

    def step(c):
        c.write(kx, vx, slots)
        qr = c.norm_rope_write(qx, kx, vx, slots, pos, freq, w, w, interleaved=True, dtype=torch.float16)
        k, v = c.read(tab, pk, 800, dtype=torch.float16)
        return (*q.head_norm_rope(qx, kx, pos, freq, w, None, eps=1e-5, dtype=torch.float32), qr, k, v,
                c.attend(qr, tab, n), c.attend(qr, tab, n, scale=0.5, max_length=300), q.attend_prompt(qr, k, v, ps, pk, scale=0.2),
                q.attend_prompt(qr, k, v, ps, pk, causal=False), c.read(tab, pk, 800)[0], c.k, c.v, c.k_scales, c.v_scales)

    native = step(c)
    monkeypatch.setattr(attention, "_calls", None)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(native, step(other), strict=True))


def test_refusals_on_the_device():
    def refused(text, fn):
        with pytest.raises((ValueError, q.QmmError), match=text):
            fn()

    def z(*shape, dtype=torch.float16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    x, w, pos, freq = z(5, 4, 32), z(32, dtype=torch.float32), i32([0] * 5), z(16, dtype=torch.float32)
    refused("k has shape", lambda: q.head_norm_rope(x, z(4, 4, 32), None, None))
    refused("k has shape", lambda: q.head_norm_rope(x, z(5, 4, 16), None, None))
    refused("k has dtype", lambda: q.head_norm_rope(x, x.float(), None, None))
    refused("contiguous last axis", lambda: q.head_norm_rope(z(5, 4, 64)[..., ::2], x, None, None))
    refused("needs positions", lambda: q.head_norm_rope(x, x, None, freq))
    refused("positions has 4", lambda: q.head_norm_rope(x, x, pos[:4], freq))
    refused("positions has dtype", lambda: q.head_norm_rope(x, x, pos.long(), freq))
    refused("inv_freq has dtype", lambda: q.head_norm_rope(x, x, pos, freq.half()))
    refused("inv_freq must be contiguous", lambda: q.head_norm_rope(x, x, pos, z(32, dtype=torch.float32)[::2]))
    refused("R=34", lambda: q.head_norm_rope(x, x, pos, z(17, dtype=torch.float32)))
    refused("R=4 ", lambda: q.head_norm_rope(x, x, pos, z(2, dtype=torch.float32)))
    refused("q_weight has 16", lambda: q.head_norm_rope(x, x, None, None, w[:16], w))
    refused("k_weight has dtype", lambda: q.head_norm_rope(x, x, None, None, w, w.half()))
    refused("q_weight has dtype", lambda: q.head_norm_rope(x, x, None, None, w.double(), w))
    refused("eps", lambda: q.head_norm_rope(x, x, None, None, w, w, eps=-1.0))
    refused("dtype", lambda: q.head_norm_rope(x, x, None, None, dtype=torch.float64))
    refused("D=24", lambda: q.head_norm_rope(z(5, 4, 24), z(5, 4, 24), None, None))
    for shape, text in (((4, 2, 24, 32), "power of two"), ((4, 2, 8, 32), "page=8"), ((4, 2, 16, 40), "D=40"), ((4, 2, 16, 272), "D=272")):
        refused(text, lambda: q.KVCache(z(*shape), z(*shape)))
    flat = z(4 * 2 * 16 * 32 + 4)
    refused("16-byte", lambda: q.KVCache(flat[4:].view(4, 2, 16, 32), z(4, 2, 16, 32)))
    refused("must be contiguous", lambda: q.KVCache(z(4, 16, 2, 32).transpose(1, 2), z(4, 2, 16, 32)))
    c = q.KVCache.empty(4, 16, 2, 32, torch.float16)
    k = z(5, 2, 32)
    refused("the cache has 2 of 32", lambda: c.write(x, x, pos))
    refused("v has shape", lambda: c.write(k, z(4, 2, 32), pos))
    refused("slots has 4", lambda: c.write(k, k, pos[:4]))
    refused("slots has dtype", lambda: c.write(k, k, pos.long()))
    refused("slots must be a device", lambda: c.write(k, k, pos.cpu()))
    refused("the cache has torch.float16", lambda: c.norm_rope_write(x, k, k, pos, None, None, dtype=torch.bfloat16))
    refused("k has dtype", lambda: c.norm_rope_write(x, k.float(), k.float(), pos, None, None))
    table, n = i32(range(4)).view(2, 2), i32([3, 3])
    refused("the cache has 2 of 32", lambda: c.attend(z(2, 3, 32), table, n))
    refused("the cache has 2 of 32", lambda: c.attend(z(2, 4, 16), table, n))
    refused("the cache has torch.float16", lambda: c.attend(z(2, 4, 32, dtype=torch.bfloat16), table, n))
    refused("table has 2 rows", lambda: c.attend(z(3, 4, 32), table, i32([1, 1, 1])))
    refused("lengths has 3", lambda: c.attend(z(2, 4, 32), table, i32([1, 1, 1])))
    refused("out has shape", lambda: c.attend(z(2, 4, 32), table, n, out=z(2, 4, 16)))
    refused("out must have q's dtype", lambda: c.attend(z(2, 4, 32), table, n, out=z(2, 4, 32, dtype=torch.bfloat16)))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused("scale", lambda: c.attend(z(2, 4, 32), table, n, scale=scale))
        refused("scale", lambda: q.attend_prompt(x, x, x, i32([0, 5]), scale=scale))
    refused("negative", lambda: c.read(table, i32([0, 1, 2]), -1))
    refused("two tensors", lambda: c.read(table, i32([0, 1, 2]), 2, out=(z(2, 2, 32), z(2, 2, 32).float())))
    refused("k has 3 heads", lambda: q.attend_prompt(x, z(5, 3, 32), z(5, 3, 32), i32([0, 5])))
    refused("v has shape", lambda: q.attend_prompt(x, k, z(5, 1, 32), i32([0, 5])))
    refused("need k_starts", lambda: q.attend_prompt(x, z(7, 2, 32), z(7, 2, 32), i32([0, 5])))
    refused("k_starts has 3", lambda: q.attend_prompt(x, k, k, i32([0, 5]), i32([0, 2, 5])))
    wide = z(5, 2 * 32 + 8)
    refused("16-byte", lambda: q.attend_prompt(x, wide[:, 4:68].unflatten(1, (2, 32)), k, i32([0, 5])))
    refused("token stride", lambda: q.attend_prompt(x, z(1, 2, 32).expand(5, 2, 32), k, i32([0, 5])))
    got = q.attend_prompt(x, k[:, :1].expand(5, 2, 32), k, i32([0, 5]))  # heads may share their rows
    assert got.shape == x.shape
