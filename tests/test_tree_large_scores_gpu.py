"""Attention of drafted tokens with scores so large that fp32 numbers of their size are many units
apart: the probabilities depend on differences, which are exact. By one launch (a cluster a unit),
by two, and with two row tiles."""
import math

import pytest
import torch

from draft_util import draft_cache

pytestmark = pytest.mark.gpu

# pages of 16: 4096 tokens take one launch at most, 9600 two
FORMS = [(5, 2, None), (5, 2, 600), (140, 1, None)]


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def check(c, o, lse, weights, top, what):
    """Chains: drafted token i of sequence b sees tokens [0, base + i]. weights[b] [n]: their
    probabilities times any number; top[b] [n]: the LSE of the first t + 1 of them."""
    T = o.shape[1]
    half = torch.finfo(c.dtype).eps / 2
    small = 2.0 ** -36 if c.dtype == torch.float16 else 0.0
    o, lse = o.double(), lse.double()
    for b, n in enumerate(c.lens):
        pg, row = c.rows(c.table, b, n)
        v, w = c.v[pg, row, 0].double(), weights[b][:, None].cuda()
        see = slice(n - T, n)
        total = w.cumsum(0)[see]
        want = ((w * v).cumsum(0)[see] / total)[:, None]
        size = ((w * v.abs()).cumsum(0)[see] / total)[:, None]
        # the output's rounding and P's; fp16 holds P down to 2^-36 of the largest; sums in 32 bits
        bound = half * want.abs() + (half + 2.0 ** -15) * size + small * v.abs().sum(0)
        assert torch.isfinite(o[b]).all(), what
        assert ((o[b] - want).abs() <= bound).all(), what
        z = top[b][see].cuda()
        # scale * log2(e), the product with the maximum, the sum and ln(2): a step each
        assert ((lse[b] - z).abs() <= z.abs() * 2.0 ** -22 + 2.0 ** -19).all(), what


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hq,width", FORMS)
def test_equal_scores(T, Hq, width, dtype):
    """From 2^9 to 2^33 (log2 units), where a step of fp32 is up to 512: O is the mean of the
    values."""
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([100, 700], [T, T], 16, 1, 64, dtype, seed=11, max_pages=width)
    q = torch.zeros((2, T, Hq, 64), dtype=c.dtype, device="cuda")
    q[..., 0] = 2.0 ** 15
    for b, n in enumerate(c.lens):
        pg, row = c.rows(c.table, b, n)
        c.k[pg, row] = 0
        c.k[pg, row, :, 0] = 2.0 ** 15
    ones = [torch.ones(n, dtype=torch.float64) for n in c.lens]
    for e in range(-21, 3):
        for sign in (1.0, -1.0):
            scale = float(torch.tensor(sign * 0.7 * 2.0 ** e, dtype=torch.float32))
            o, lse = fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, scale=scale)
            check(c, o, lse, ones, [scale * 2.0 ** 30 + x.cumsum(0).log() for x in ones], (e, sign))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hq,width", FORMS)
@pytest.mark.parametrize("growth", [1.7, 3.3, 4.7, 9.1])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_maximum_that_grows(T, Hq, width, dtype, growth, sign):
    """By `growth` log2 units from one tile of 128 tokens to the next, on top of 2^23 times as much:
    products of q and k that fp32 holds exactly, so that the differences are known."""
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([1500, 390], [T, T], 16, 1, 64, dtype, seed=5, max_pages=width)
    q = torch.zeros((2, T, Hq, 64), dtype=c.dtype, device="cuda")
    q[..., 0], q[..., 1] = 2.0 ** 12, 1.0
    scale = float(torch.tensor(growth * math.log(2.0), dtype=torch.float32))
    weights, top = [], []
    for b, n in enumerate(c.lens):
        pg, row = c.rows(c.table, b, n)
        step = torch.arange(n) // 128
        c.k[pg, row] = 0
        c.k[pg, row, :, 0] = sign * 2.0 ** 11
        c.k[pg, row, 0, 1] = (sign * step).to(c.dtype).cuda()
        s = scale * (step - step.max()).double()
        weights.append(s.exp())
        top.append(scale * (2.0 ** 23 + float(step.max())) + s.logcumsumexp(0))
    o, lse = fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, scale=sign * scale)
    check(c, o, lse, weights, top, growth)
