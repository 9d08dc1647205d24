"""paged_accept of chains, whose parents need not be written out."""
import pytest
import torch

from draft_util import draft_cache
from test_pool_gpu import int32


def test_the_number_of_drafted_tokens_is_asked_for():
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([5], [3], 16, 2, 64, "bf16", device="cpu")
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="T has to be given"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, one)
    with pytest.raises(ValueError, match="T has to be given"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, one, None)
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, one, T=3)
    parents = torch.full((1, 3), -1, dtype=torch.int32)
    with pytest.raises(ValueError, match="parents"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, one, parents, T=4)
    with pytest.raises(ValueError, match="T is out of range"):
        fa.paged_accept(c.k.cuda() if torch.cuda.is_available() else c.k, c.v, c.table, c.seqlens, one,
                        T=2 ** 32 + 3)


@pytest.mark.gpu
@pytest.mark.parametrize("side", [False, True])
def test_a_chain_without_parents(side):
    """As with the chain's parents: path, lengths, rows and weights."""
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    T, new, leaf = 6, [6, 0, 3, 6], [5, -1, 1, -1]
    parents = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(4, 1)
    stream = torch.cuda.Stream() if side else None
    got = []
    for p, kw in ((parents, {}), (None, dict(T=T)), (parents, dict(T=T))):
        c = draft_cache([30, 5, 9, 40], new, 16, 2, 64, "fp16", weights=True)
        torch.cuda.synchronize()
        path, lens = fa.paged_accept(c.k, c.v, c.table, c.seqlens, int32(leaf), p, new_lens=int32(new),
                                     weights=c.w, stream=stream, **kw)
        torch.cuda.synchronize()
        got.append([path, lens, c.k, c.v, c.w])
    assert got[0][0].tolist() == [[0, 1, 2, 3, 4, 5], [-1] * 6, [0, 1, -1, -1, -1, -1], [-1] * 6]
    assert got[0][1].tolist() == [36, 5, 11, 40]
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert x.dtype == y.dtype and torch.equal(x.nan_to_num(), y.nan_to_num())
    assert fa.device_error() == 0
    for bad in (0, 1025):
        with pytest.raises(fa.FaError):
            fa.paged_accept(c.k, c.v, c.table, c.seqlens, int32(leaf), T=bad)
