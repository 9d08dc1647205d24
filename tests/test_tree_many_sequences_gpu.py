"""Attention of drafted tokens for the largest batches: the lengths that a CTA reads before its run
starts, and units of nothing but padding, take longer than any wait on a tile may."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [1, 2])   # one launch that clears the padding itself, and two
def test_sequences_without_drafted_tokens(width):
    """2^26 sequences of one query, the last five of them with a drafted token: three seconds."""
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    B, d, live = 1 << 26, 64, 5
    q = torch.ones((B, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((2, 128, 1, d), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    new[B - live:] = 1
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, 1, 1), float("nan"), device="cuda")
    fa.paged_tree_attention(q, k, k * 3, table, lens, new_lens=new, scale=1 / 64, out=o, lse=lse)
    assert fa.device_error() == 0
    assert (o[B - live:] == 3).all() and (lse[B - live:] == 1).all()
    assert not o[:B - live].any() and torch.isneginf(lse[:B - live]).all()
    del q, o
    torch.cuda.empty_cache()
