"""The paged cache as its documentation uses it."""
import os
import re

import pytest
import torch

from paged_util import (Cache, check_decode, decode_ref, default_scale, evict_ref, key_weights_ref,
                        same_bits)

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


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2)])
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


@pytest.mark.parametrize("Hq,Hkv,d,dtype,page", [(8, 2, 128, "bf16", 16), (6, 1, 64, "fp16", 64)])
def test_prompt_with_shared_key_heads(Hq, Hkv, d, dtype, page):
    """A padded prompt whose query heads share key heads: the forward over K and V repeated for
    every query head, key weights and pages of the key heads alone, decoding steps, an eviction
    into free pages, and steps over those."""
    import io_aware_attention_fa2_gb300 as fa
    B, N, G = 2, 301, Hq // Hkv
    lens, budget, recent = [301, 120], 150, 30
    width = -(-(N + 16) // page)
    c = Cache([0, 0], page, Hkv, d, dtype, seed=Hq, weights=True, max_pages=width,
              spare=4 * width)
    c.table, free = (x.cuda().contiguous() for x in c.free[:4 * width].view(2, 2, width))
    q = torch.randn((B, N, Hq, d), generator=c.g).to(c.dtype).cuda()
    k, v = (torch.randn((B, N, Hkv, d), generator=c.g).to(c.dtype).cuda() for _ in range(2))
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward(q, k.repeat_interleave(G, 2), v.repeat_interleave(G, 2),
                                  causal=True, seqlens_k=lens_t)
    w = fa.key_weights(q, k, lse, causal=True, seqlens_k=lens_t)
    ref, bound = key_weights_ref(q, k, lse, default_scale(d), True, (-1, -1), lens)
    assert ((w.double().cpu() - ref).abs() <= bound).all()
    # the probabilities of every query sum to one over its keys, for each of its heads
    assert (w.sum(-1).cpu() - G * torch.tensor(lens)[:, None]).abs().max() < G * N * 2.0 ** -10
    fa.fa_paged_append(k, v, c.k, c.v, c.table, lens_t, new_lens=lens_t, w=w, weights=c.w)
    c.lens, c.seqlens = list(lens), lens_t.clone()
    last = torch.stack([q[b, lens[b] - 1] for b in range(B)])
    o1, lse1 = fa.paged_attention(last, c.k, c.v, c.table, c.seqlens)
    ref = decode_ref(c, last, default_scale(d))
    check_decode(c, last, o1, lse1, ref, "prompt")
    want = torch.stack([o[b, lens[b] - 1] for b in range(B)]).double().cpu()
    assert ((o1.double().cpu() - want).abs() <= 2 * ref[3]).all()

    def steps(n):
        for _ in range(n):
            c.lens = [x + 1 for x in c.lens]
            c.seqlens += 1
            new = [torch.randn((B, 1, Hkv, d), generator=c.g).to(c.dtype).cuda() for _ in range(2)]
            fa.fa_paged_append(*new, c.k, c.v, c.table, c.seqlens, weights=c.w)
            query = c.query(Hq)
            got = fa.paged_attention(query, c.k, c.v, c.table, c.seqlens, weights=c.w)
            check_decode(c, query, *got, decode_ref(c, query, default_scale(d)), c.lens)

    steps(3)
    ref = evict_ref(c, free, budget, recent)
    kept, c.seqlens = fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, free, budget, recent)
    assert torch.equal(kept.cpu(), ref[0]) and torch.equal(c.seqlens.cpu(), ref[1])
    assert same_bits(c.k, ref[2]) and same_bits(c.v, ref[3]) and same_bits(c.w, ref[4])
    c.table, c.lens = free, ref[1].tolist()
    steps(3)
