"""The paged cache as its documentation uses it."""
import os
import re

import pytest
import torch

from paged_util import Cache, check_decode, decode_ref, default_scale

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def example(path, word):
    """The Python block of a Markdown file that contains `word`."""
    text = open(os.path.join(ROOT, path)).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if word in b]
    assert len(blocks) == 1
    return blocks[0]


@pytest.mark.parametrize("Hq,Hkv", [(2, 2)])
def test_readme_example_and_a_step_after_it(Hq, Hkv):
    """The README's block as it stands, then one more decoding step with the names it leaves: the
    attention over the tokens that the eviction kept, head by head."""
    import io_aware_attention_fa2_gb300 as fa
    B, N, d, page, budget = 2, 4300, 64, 64, 4096
    g = torch.Generator().manual_seed(Hq)

    def randn(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()

    width = N // page + 1
    pages = torch.randperm(2 * B * width, generator=g).to(torch.int32).cuda().view(2, B, width)
    ns = dict(q=randn(B, N, Hq, d), k=randn(B, N, Hkv, d), v=randn(B, N, Hkv, d),
              q1=randn(B, Hq, d), k1=randn(B, 1, Hkv, d), v1=randn(B, 1, Hkv, d),
              k_pages=torch.zeros((2 * B * width, page, Hkv, d), dtype=torch.bfloat16,
                                  device="cuda"),
              weights=torch.zeros((2 * B * width, Hkv, page), device="cuda"), Hq=Hq, Hkv=Hkv,
              block_table=pages[0].contiguous(), free_pages=pages[1].contiguous(),
              seqlens=torch.full((B,), N, dtype=torch.int32, device="cuda"))
    ns["v_pages"] = torch.zeros_like(ns["k_pages"])
    exec(example("README.md", "paged_evict"), ns)
    assert ns["kept"].shape == (B, Hkv, budget) and ns["seqlens"].tolist() == [budget] * B
    q2 = randn(B, Hq, d)
    o, lse = fa.paged_attention(q2, ns["k_pages"], ns["v_pages"], ns["block_table"], ns["seqlens"])
    K, V = (torch.cat([ns[x], ns[x + "1"]], 1) for x in "kv")
    c = Cache([budget] * B, page, Hkv, d, "bf16")      # the kept tokens, in pages of their own
    kept = ns["kept"].long()
    for b in range(B):
        pg, row = c.rows(c.table, b, budget)
        for h in range(Hkv):
            c.k[pg, row, h], c.v[pg, row, h] = K[b, kept[b, h], h], V[b, kept[b, h], h]
    check_decode(c, q2, o, lse, decode_ref(c, q2, default_scale(d)), "after the README's block")
