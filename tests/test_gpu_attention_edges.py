"""Head norms, the paged cache and attention where their ranges end, and what may stand beside a row: on the device, against
the fp64 oracle or bit for bit."""

import numpy as np
import pytest
import torch

import block_quantized_weight_matmul_amd as q
from tests.test_gpu_attention import attend_reference, i32, within
from tests.test_gpu_f8 import dev

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
