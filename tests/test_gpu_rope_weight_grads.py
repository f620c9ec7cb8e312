"""The norm weights' gradients of qk_norm_rope_bwd where many rows are summed, against 64 bits, with a bound that counts
the kernel's own chain of additions and that a missing part of the rows does not pass."""
import pytest
import torch

import plain64 as P
from plain64 import gen, randn
from test_gpu_rope import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import long_context_mqa_b200 as m
    return m


def chain(T, heads, d, blocks):
    """Additions in a row at most, on the way from a row to the sum: a lane's rows (every warp of `blocks` blocks of four
    takes items, a run of a token's passes each: with p warps a token ceil(T p / warps) items of ceil(n / p) of its n passes,
    p <= n, which is at most 2 T n / warps + n + 1), two shuffles, four warps, the records of a strip, 32 strips."""
    rows = 256 // d
    n = sum(-(-h // rows) for h in heads)
    return 2 * T * n // (4 * blocks) + n + 1 + 2 + 4 + -(-blocks // 32) + 32


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(40001, 3, 1, 64, 32), (2500, 8, 1, 128, 64), (9000, 64, 1, 128, 128), (20000, 5, 5, 64, 64),
                                           (1009, 32, 4, 64, 64), (300, 64, 8, 128, 128)])
def test_weight_gradients_of_many_rows(hs2, T, Hq, Hk, d, rot, interleaved):
    q, k, _, pos, freq, (qw, kw) = inputs(T, Hq, Hk, d, rot, torch.float32, first=5)
    g = gen(9)
    gq, gk = randn(g, T, Hq, d), randn(g, T, Hk, d, dtype=torch.float32, std=4.0)
    got = hs2.qk_norm_rope_bwd(q, k, pos, freq, gq, gk, q_weight=qw, k_weight=kw, interleaved=interleaved)
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    for x, w, dy, dw, name in ((q, qw, gq, got[2], "q"), (k, kw, gk, got[3], "k")):
        # the terms g x r of every row (plain64's formulas)
        cos, sin = P.turns(pos, freq, d, rot, interleaved, 1.0)
        y, xd = dy.double(), x.double()
        back = y * cos - P.partner(y * sin, rot, interleaved)
        r = 1 / (xd.square().mean(-1, keepdim=True) + P.EPS).sqrt()
        terms = (back * xd * r).sum(1)  # [T, d]
        size = ((y.abs() + P.partner(y, rot, interleaved).abs()) * xd.abs() * r).sum((0, 1))
        want = terms.sum(0)
        bound = (2.0 ** -18 + chain(T, (Hq, Hk), d, blocks) * 2.0 ** -24) * size + 2.0 ** -24 * want.abs()
        P.near(dw, want, bound, f"d{name}_weight")
        # the bound tells: zeros are outside in nearly every column, a sum without one block's tokens in most
        terms, bound, want = terms.cpu(), bound.cpu(), want.cpu()
        assert float((want.abs() > bound).double().mean()) > 0.9
        part = terms[torch.arange(T) % (4 * blocks) < 4].sum(0)
        assert float((part.abs() > bound).double().mean()) > 0.5, (name, float((part.abs() / bound).median()))
