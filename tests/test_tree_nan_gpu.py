"""Attention of drafted tokens: what is not a number in a live query or in a key that is seen
reaches the result, and so does an infinite value behind a score of minus infinity, on tables of
any width: by one launch (a cluster a unit), by two, and with two row tiles."""
import math

import pytest
import torch

from draft_util import check_tree, draft_cache, random_trees, tree_ref
from paged_util import default_scale

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def run(c, q, parents):
    import io_aware_attention_fa2_gb300 as fa
    o, lse = fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, parents=parents.cuda())
    return o.cpu(), lse.cpu()


def queries(c, B, T, Hq):
    return torch.randn((B, T, Hq, c.d), generator=c.g).to(c.dtype).cuda()


def check_rows(o, lse, ref, keep, what):
    """The rows (b, i, h) of `keep` within the bounds of the definition."""
    rows = lambda x: x[keep]                                 # noqa: E731  [B, T, Hq, d]
    heads = lambda x: x.transpose(1, 2)[keep]                # noqa: E731  [B, Hq, T]
    check_tree(rows(o), heads(lse), (rows(ref[0]), heads(ref[1]), rows(ref[2]), heads(ref[3])), what)


# pages of 16: 4096 tokens take one launch at most, 9600 two
WIDTHS = [(6, 4, 2, None), (6, 4, 2, 600), (130, 2, 1, None)]


@pytest.mark.parametrize("T,Hq,Hkv,width", WIDTHS)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_queries_that_are_not_finite(T, Hq, Hkv, width, d, dtype, bad):
    """One number of one query: all of its row's scores are NaN, or infinite of both signs, so that
    O is NaN and LSE not finite; the other rows are as ever."""
    c = draft_cache([300, 1000], [T, T], 16, Hkv, d, dtype, seed=T, max_pages=width)
    q, parents = queries(c, 2, T, Hq), random_trees(c.g, 2, T)
    ref = tree_ref(c, q, default_scale(d), parents)
    keep = torch.ones((2, T, Hq), dtype=torch.bool)
    for b, i, h in ((0, 2, Hq - 1), (1, T - 1, 0), (1, 0, Hq - 1)):
        q[b, i, h, d - 3] = bad
        keep[b, i, h] = False
    o, lse = run(c, q, parents)
    assert torch.isnan(o[~keep]).all()
    bad_lse = lse.transpose(1, 2)[~keep]
    assert torch.isnan(bad_lse).all() if math.isnan(bad) else not torch.isfinite(bad_lse).any()
    check_rows(o, lse, ref, keep, (T, bad))


@pytest.mark.parametrize("T,Hq,Hkv,width", WIDTHS)
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("ctx", [127, 255, 1023])
def test_a_nan_key_alone_in_a_tile(T, Hq, Hkv, width, d, dtype, ctx):
    """Drafted token 3 sees only itself of the last tile, and its key is NaN: so are O and LSE of its
    rows. The others do not see it."""
    c = draft_cache([ctx], [T], 16, Hkv, d, dtype, seed=ctx, max_pages=width)
    q, parents = queries(c, 1, T, Hq), torch.full((1, T), -1, dtype=torch.int32)
    ref = tree_ref(c, q, default_scale(d), parents)
    c.k[int(c.table[0, (ctx + 3) // 16]), (ctx + 3) % 16] = NAN
    o, lse = run(c, q, parents)
    keep = torch.ones((1, T, Hq), dtype=torch.bool)
    keep[0, 3] = False
    assert torch.isnan(o[~keep]).all() and torch.isnan(lse[0, :, 3]).all()
    check_rows(o, lse, ref, keep, ctx)


@pytest.mark.parametrize("T,Hq,Hkv,width", WIDTHS)
@pytest.mark.parametrize("where", [0, 130, 299])
def test_a_nan_key_of_the_context(T, Hq, Hkv, width, where):
    """Every row of the key head that has it sees it."""
    c = draft_cache([300], [T], 16, Hkv, 64, "bf16", seed=where, max_pages=width)
    q, parents = queries(c, 1, T, Hq), random_trees(c.g, 1, T)
    ref = tree_ref(c, q, default_scale(64), parents)
    c.k[int(c.table[0, where // 16]), where % 16, 0, 7] = NAN
    o, lse = run(c, q, parents)
    keep = torch.ones((1, T, Hq), dtype=torch.bool)
    keep[:, :, :Hq // Hkv] = False
    assert torch.isnan(o[~keep]).all() and torch.isnan(lse.transpose(1, 2)[~keep]).all()
    if keep.any():
        check_rows(o, lse, ref, keep, where)


@pytest.mark.parametrize("T,Hq,Hkv,width", WIDTHS)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_an_infinite_value_behind_a_score_of_minus_infinity(T, Hq, Hkv, width, d, dtype):
    """Alone in the last tile, too: 0 times infinity is no finite number; the other columns, and LSE,
    are those without the token."""
    ctx = 255
    c = draft_cache([ctx], [T], 16, Hkv, d, dtype, seed=d, max_pages=width)
    q, parents = queries(c, 1, T, Hq), torch.full((1, T), -1, dtype=torch.int32)
    q[0, 3, :, 0] = 1.0
    pg, row = int(c.table[0, (ctx + 3) // 16]), (ctx + 3) % 16
    ref = tree_ref(c, q, default_scale(d), parents, drop=lambda b, t: t == ctx + 3)
    c.k[pg, row, :, 0] = -INF
    c.v[pg, row, :, 1] = INF
    o, lse = run(c, q, parents)
    assert not torch.isfinite(o[0, 3, :, 1]).any()
    o[0, 3, :, 1] = ref[0][0, 3, :, 1].to(o.dtype)
    check_tree(o, lse, ref, "behind")
