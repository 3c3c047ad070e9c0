"""Head norms, the paged cache and attention where their ranges end, and what may stand beside a row: on the device, against
the fp64 oracle or bit for bit."""

import struct

import numpy as np
import pytest
import torch

import block_quantized_weight_matmul_amd as q
from block_quantized_weight_matmul_amd import _lib as L
from tests.test_gpu_attention import CACHES, attend_reference, filled, frequencies, i32, within
from tests.test_gpu_f8 import DTYPES, dev

pytestmark = pytest.mark.gpu


def test_join_of_more_than_2_23_heads():
    """More heads in all than the join's grid has workgroups along x: its surplus ones touch nothing."""
    g = np.random.default_rng(101)
    B, Hq, D, page, W = 32769, 257, 16, 4096, 5
    assert B * Hq > 1 << 23
    c = q.KVCache.empty(W, page, 1, D, torch.float16)
    k, v = (dev(g.standard_normal((W * page, 1, D))) for _ in "kv")
    c.write(k, v, i32(range(W * page)))
    table = np.tile(g.permutation(W).astype(np.int32), (B, 1))
    # three pieces: sequences that have all of them at both ends and in the middle, all others a few tokens or none
    lengths = np.arange(B) % 4
    some = [0, 1, 2, 3, B // 2, B - 1]
    lengths[[0, B // 2, B - 1]] = W * page, 7000, W * page - 1
    qx = dev(g.standard_normal((1, Hq, D)), torch.float16).expand(B, Hq, D)
    room = torch.full((B * Hq * D + (1 << 25),), 9.0, device="cuda", dtype=torch.float16)
    out = room[1 << 24:-(1 << 24)].view(B, Hq, D)
    c.attend(qx, dev(table, torch.int32), dev(lengths, torch.int32), out=out)
    assert bool((room[:1 << 24] == 9).all()) and bool((room[-(1 << 24):] == 9).all())
    ref, bound = attend_reference(c, table[some], lengths[some], qx[some], D ** -0.5)
    within(out[some], ref, bound)
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[some] = False
    for n in range(4):  # of one length: the same bits
        rows = out[dev(lengths == n, torch.bool) & rest]
        assert torch.equal(rows, out[n or 4].expand_as(rows))


@pytest.mark.parametrize("D", [32, 128, 256])
def test_a_token_of_zeros_leaves_its_neighbours_bits(D):
    """Without eps, a token of zeros takes the root's other form; the tokens that share its wave do not."""
    g = np.random.default_rng([102, D])
    x = dev(g.standard_normal((64, 4, D)) * 2)
    w = dev(1 + 0.2 * g.standard_normal(D))
    want = q.head_norm_rope(x, x, None, None, w, w, eps=0.0)
    spoiled = x.clone()
    spoiled[::4] = 0
    spoiled[1::8, 2] = 1e-18  # a mean square below 2^-100
    keep = (spoiled == x).all(2)
    for a, b in zip(want, q.head_norm_rope(spoiled, spoiled, None, None, w, w, eps=0.0)):
        assert torch.equal(a[keep], b[keep])


def alone(n, at, Hq, H, D, dtype, g):
    """Queries, keys and values of one sequence in which the scores of token `at` and later ones can be raised, whatever the query:
    a column of ones meets what the keys hold there."""
    qx = g.standard_normal((n, Hq, D)) * 1.5
    qx[..., 3] = 1.0
    k, v = g.standard_normal((2, n, H, D))
    k[..., 3] = 0.0
    return dev(qx, dtype), dev(k, dtype), dev(v, dtype)


PREFIXES = [(300, 205, 2, 1, 48), (300, 205, 2, 1, 128), (300, 205, 2, 1, 256), (70, 33, 8, 2, 128), (1100, 1000, 8, 2, 64), (129, 100, 3, 3, 96),
            (900, 515, 16, 4, 128), (400, 70, 1, 1, 32), (200, 199, 4, 2, 192)]


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,at,Hq,H,D", PREFIXES)
def test_prompt_rows_keep_their_bits_whatever_follows(n, at, Hq, H, D, t):
    """Keys and values that come after a query do not change a bit of its output: not by how large their scores are (a maximum
    that moves by much or by little, scores past 2^20), nor by their values."""
    g = np.random.default_rng([103, n, D])
    qx, k, v = alone(n, at, Hq, H, D, t, g)
    s = i32([0, n])
    for scale in (D ** -0.5, 0.0625):
        want = q.attend_prompt(qx, k, v, s, scale=scale)
        # scores higher by 12 (2^17 and more), by 100, and past 2^20
        for raised in (12 / scale, 100 / scale, 6e4, *([2.0 ** 30] if t == torch.bfloat16 else [])):
            k2, v2 = k.clone(), v.clone()
            k2[at:, :, 3] = raised
            k2[at + 1::2, :, 3] *= -1
            v2[at:] *= -3
            got = q.attend_prompt(qx, k2, v2, s, scale=scale)
            assert torch.equal(got[:at], want[:at]), (scale, raised)
            assert not torch.equal(got[at:], want[at:])
    # rows whose own scores are past 2^20, beside rows whose are not
    if t == torch.bfloat16:
        far = qx.clone()
        far[::3] *= 2.0 ** 24
        some = torch.ones(n, dtype=torch.bool)
        some[::3] = False
        got, want = q.attend_prompt(far, k, v, s), q.attend_prompt(qx, k, v, s)
        assert torch.equal(got[some], want[some])


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,at,Hq,H,D", PREFIXES)
def test_prompt_rows_keep_their_bits_before_infinities(n, at, Hq, H, D, t):
    """The same for infinite and NaN keys and values; what does not see the column keeps its bits too."""
    g = np.random.default_rng([104, n, D])
    qx, k, v = alone(n, at, Hq, H, D, t, g)
    s = i32([0, n])
    want = q.attend_prompt(qx, k, v, s)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for rows in (slice(at, at + 1), slice(at, None, 3), slice(at, None)):
            k2, v2 = k.clone(), v.clone()
            k2[rows, H - 1, 5] = bad
            assert torch.equal(q.attend_prompt(qx, k2, v, s)[:at], want[:at])
            v2[rows, H - 1, 5] = bad
            got = q.attend_prompt(qx, k, v2, s)
            assert torch.equal(got[:at], want[:at])
            other = torch.ones((Hq, D), dtype=torch.bool)
            other[Hq - Hq // H:, 5] = False
            assert torch.equal(got[:, other], want[:, other])
            assert not bool(torch.isfinite(got[at:, ~other]).any())
        v2 = v.clone()
        v2[at:] = bad
        assert torch.equal(q.attend_prompt(qx, k, v2, s)[:at], want[:at])


def limit_of(v, weights):
    """The definition's outputs where values [m] are infinite or NaN and all weights [n, m] are 0 or well above it."""
    with np.errstate(invalid="ignore"):
        return np.array([sum((w * x for w, x in zip(row, v) if w), 0.0) for row in weights])


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,H", [(100, 1), (700, 8)])
def test_prompt_infinite_values_that_are_seen(n, H, t):
    """With equal scores: an infinity of one sign is the output, two signs or a NaN are NaN."""
    g = np.random.default_rng([105, n])
    D = 64
    v = g.standard_normal((n, H, D))
    v[n // 4, :, 3] = np.inf
    v[n // 2, :, 4], v[n // 2 + 3, :, 4] = -np.inf, -np.inf
    v[n // 3, :, 5], v[n - 9, :, 5] = -np.inf, np.inf
    v[0, :, 6] = np.nan
    z = torch.zeros((n, H, D), device="cuda", dtype=t)
    got = q.attend_prompt(z, z, dev(v, t), i32([0, n])).double().cpu().numpy()
    for column in (3, 4, 5, 6):
        want = limit_of(v[:, 0, column], np.tri(n))
        spoiled = ~np.isfinite(want)
        assert spoiled.any()
        for h in range(H):
            assert np.array_equal(got[spoiled, h, column], want[spoiled], equal_nan=True), column
            assert np.isfinite(got[~spoiled, h, column]).all()


ONE_KIND = [([40], 1), ([100, 33], 2), ([500], 8), ([260] * 40, 8), ([3000, 700], 1), ([5000], 2)]  # lengths, key heads


@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("lengths,H", ONE_KIND)
def test_decode_infinite_values(lengths, H, kind, D):
    """With equal scores: an infinity of one sign is the output, two signs or a NaN are NaN, and the columns beside them keep
    their bits, however the work is divided."""
    g = np.random.default_rng([106, len(lengths), D])
    c, table, owner, tok = filled(g, lengths, 16, H, D, kind)
    slots = i32(table[owner, tok // 16] * 16 + tok % 16)
    tab, n = i32(table.flatten()).view(len(lengths), -1), i32(lengths)
    k, v = torch.zeros((len(tok), H, D), device="cuda"), g.standard_normal((len(tok), H, D))
    qx = torch.zeros((len(lengths), 2 * H, D), device="cuda", dtype=c.dtype)
    bounds = (None, 0, 5000)
    c.write(k, dev(v), slots)
    want = [c.attend(qx, tab, n, max_length=m) for m in bounds]
    for b, m in enumerate(lengths):
        first = int(np.flatnonzero(owner == b)[0])
        v[first + m // 4, :, 3] = np.inf
        v[[first + m // 2, first + m // 2 + 3], :, 4] = -np.inf
        v[first + m // 3, :, 5], v[first + m - 9, :, 5] = -np.inf, np.inf
        v[first, :, 6] = np.nan
    c.write(k, dev(v), slots)
    others = [i for i in range(D) if not 3 <= i <= 6]
    for m, y in zip(bounds, want):
        got = c.attend(qx, tab, n, max_length=m)
        assert bool((got[..., 3] == float("inf")).all()) and bool((got[..., 4] == -float("inf")).all())
        assert bool(torch.isnan(got[..., 5:7]).all())
        assert torch.equal(got[..., others], y[..., others])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_decode_infinite_values_of_any_probability(kind):
    """Probabilities from 1 down to 2^-24, at places of every kind in a tile: infinities all the same."""
    g = np.random.default_rng(107)
    H, D, m = 1, 64, 64
    c, table, _, tok = filled(g, [m], 16, H, D, kind)
    slots = i32(table[0, tok // 16] * 16 + tok % 16)
    k = np.zeros((m, H, D))
    k[:, 0, 0] = -np.linspace(0, 24, m) * np.log(2)  # scores of a query of ones, in powers of two
    v = g.standard_normal((m, H, D))
    v[np.arange(m), 0, np.arange(m)] = np.inf  # column j: token j's
    qx = torch.zeros((1, 1, D), device="cuda", dtype=c.dtype)
    qx[..., 0] = 1
    c.write(dev(k), dev(v), slots)
    got = c.attend(qx, i32(table.flatten()).view(1, -1), i32([m]), scale=1.0)
    assert bool((got == float("inf")).all())


@pytest.mark.parametrize("kind", CACHES)
def test_decode_joins_what_pieces_of_no_weight_hold(kind):
    """A NaN or infinite value in a piece whose probabilities are rounded to zero beside another piece's: seen all the same, in
    one piece or many."""
    g = np.random.default_rng(108)
    H, D, m = 1, 128, 4000
    c, table, _, tok = filled(g, [m], 16, H, D, kind)
    at = table[0, tok // 16] * 16 + tok % 16
    k, v = np.zeros((m, H, D)), g.standard_normal((m, H, D))
    k[:-100, 0, 0] = -400.0
    qx = torch.ones((1, 2, D), device="cuda", dtype=torch.float16 if kind == "e4m3" else c.dtype)
    c.write(dev(k), dev(v), i32(at))
    tab = i32(table.flatten()).view(1, -1)
    want = [c.attend(qx, tab, i32([m]), scale=1.0, max_length=bound) for bound in (None, 0)]
    assert all(bool(torch.isfinite(y).all()) for y in want)
    for bad in (float("nan"), float("inf")):
        v2 = dev(v)
        v2[50, 0, 5] = bad
        c.write(dev(k), v2, i32(at))
        for bound, y in zip((None, 0), want):
            got = c.attend(qx, tab, i32([m]), scale=1.0, max_length=bound)
            assert not bool(torch.isfinite(got[..., 5]).any())
            if kind != "e4m3":
                others = [i for i in range(D) if i != 5]
                assert torch.equal(got[..., others], y[..., others])


def test_numbers_beyond_fp32_are_refused():
    x, w = torch.zeros((5, 4, 32), device="cuda", dtype=torch.float16), torch.ones(32, device="cuda")
    c = q.KVCache.empty(4, 16, 2, 32, torch.float16)
    table, n = i32(range(4)).view(2, 2), i32([3, 3])
    for far in (1e39, -1e39, 1e300):
        for what, call in (("eps", lambda: q.head_norm_rope(x, x, None, None, w, w, eps=far)),
                           ("eps", lambda: c.norm_rope_write(x, x[:, :2], x[:, :2], i32([0] * 5), None, None, w, w, eps=far)),
                           ("scale", lambda: c.attend(x[:2], table, n, scale=far)),
                           ("scale", lambda: q.attend_prompt(x, x, x, i32([0, 5]), scale=far))):
            with pytest.raises(q.QmmError, match=what):
                call()


@pytest.mark.parametrize("kind", CACHES)
def test_table_entries_past_the_last_page(kind):
    """Whatever they hold: pages of NaN, of other sequences, or none at all."""
    g = np.random.default_rng(109)
    lengths, page, H, D = [40, 33, 0, 1500, 129], 16, 2, 64
    c, table, _, _ = filled(g, lengths, page, H, D, kind)
    B, n = len(lengths), i32(lengths)
    past = np.arange(table.shape[1])[None] >= -(-np.array(lengths) // page)[:, None]
    qx = dev(g.standard_normal((B, 4, D)), torch.float16 if kind == "e4m3" else c.dtype)
    first = i32(np.concatenate([[0], np.cumsum(lengths)]))

    def calls(entries):
        tab = i32(np.where(past, entries, table).flatten()).view(B, -1)
        return (*(c.attend(qx, tab, n, max_length=m) for m in (None, 0, 200)), *c.read(tab, first, sum(lengths)))

    want = calls(-1)
    assert all(bool(torch.isfinite(y).all()) for y in want)
    for entries in (g.integers(0, c.pages, table.shape), c.pages, (1 << 31) - 1, -(1 << 31)):
        assert all(torch.equal(a, b) for a, b in zip(calls(entries), want))


@pytest.mark.parametrize("kind", CACHES)
def test_a_page_that_is_none_among_many_pieces(kind):
    """A table entry that names no page makes its sequence's outputs NaN, in one piece or many, and no other's."""
    g = np.random.default_rng(110)
    lengths, page, H, D = [5000, 40, 3000], 16, 1, 128
    c, table, _, _ = filled(g, lengths, page, H, D, kind)
    for t in (torch.float16, torch.bfloat16) if kind == "e4m3" else (c.dtype,):
        qx = dev(g.standard_normal((3, 2, D)), t)
        for bound in (None, 0, 300):
            want = c.attend(qx, i32(table.flatten()).view(3, -1), i32(lengths), max_length=bound)
            assert bool(torch.isfinite(want).all())
            for b, at, entry in ((0, 0, -1), (0, 150, c.pages), (0, 312, -9), (1, 2, 1 << 30), (2, 187, -1), (2, 100, c.pages)):
                bad = table.copy()
                bad[b, at] = entry
                got = c.attend(qx, i32(bad.flatten()).view(3, -1), i32(lengths), max_length=bound)
                others = [i for i in range(3) if i != b]
                assert bool(torch.isnan(got[b]).all()) and torch.equal(got[others], want[others])


@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,H,D,R", [(1, 40, 13, 128, 128), (300, 9, 6, 80, 48), (40, 33, 7, 256, 256), (8192, 5, 5, 64, 16)])
def test_head_norm_in_place(T, Hq, H, D, R, t, interleaved):
    """q_out and k_out may be q and k themselves: more heads than a layer loads at once, with the bits of the call that gives
    new tensors."""
    g = np.random.default_rng([111, T, D])
    qx, kx = (dev(g.standard_normal((T, n, D)), t) for n in (Hq, H))
    w, freq, pos = dev(1 + 0.2 * g.standard_normal(D)), dev(frequencies(R)), i32(g.integers(0, 1 << 20, T))
    want = q.head_norm_rope(qx, kx, pos, freq, w, w, interleaved=bool(interleaved))
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[t]
    args = struct.pack("21q4if4x", qx.data_ptr(), kx.data_ptr(), 0, w.data_ptr(), w.data_ptr(), pos.data_ptr(), freq.data_ptr(), 0,
                       qx.data_ptr(), kx.data_ptr(), Hq * D, D, H * D, D, 0, 0, T, Hq, H, D, R, dt, 0, dt, interleaved, 1e-6)
    L.check(L.lib.qmm_head_norm_rope(args, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(qx, want[0]) and torch.equal(kx, want[1])


@pytest.mark.parametrize("bad", [0.5, float("inf"), float("nan")])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_rows_whose_scores_are_all_minus_infinity(kind, bad):
    """Keys of -inf under a query that is positive there: zeros, whatever the values are; the other queries are not touched."""
    g = np.random.default_rng(112)
    t, H, D = DTYPES[kind], 2, 64
    for n in (40, 100, 500, 4000):
        qx, k, v = g.standard_normal((n, 4, D)), g.standard_normal((n, H, D)), np.full((n, H, D), 0.5)
        qx[:, 0, 7] = 1.0                      # head 0, of key head 0
        qx[:, 1:, 7] = 0.0
        k[:, 0, 7] = -np.inf
        v[n // 2, 0, 5] = v[3, 0, 9] = bad
        qx[:, 1] = 0                           # head 1 meets 0 * -inf
        qd, kd, vd = (dev(a, t) for a in (qx, k, v))
        got = q.attend_prompt(qd, kd, vd, i32([0, n]))
        assert bool((got[:, 0] == 0).all()) and bool(torch.isnan(got[:, 1]).all())
        assert bool(((got[:, 2:].float() - 0.5).abs() < 1e-2).all())
        c, table, _, tok = filled(g, [n], 16, H, D, kind)
        c.write(kd, vd, i32(table[0, tok // 16] * 16 + tok % 16))
        for m in (None, 0, 5000):
            got = c.attend(qd[-1:], i32(table.flatten()).view(1, -1), i32([n]), max_length=m)
            assert bool((got[:, 0] == 0).all()) and bool(torch.isnan(got[:, 1]).all())
            assert bool(((got[:, 2:].float() - 0.5).abs() < 1e-2).all())
