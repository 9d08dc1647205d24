"""Drafted and branching sequences with random arguments: attention against float64, the books
against plain lists; and padding that no segment, one segment or the joining kernel writes."""
import random

import pytest
import torch

from draft_util import Pool, accept_ref, check_tree, draft_cache, line, random_trees, tree_ref
from paged_util import default_scale, same_bits

pytestmark = pytest.mark.gpu
FA_ERR_PAGE = -13


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed", range(60))
def test_tree_and_accept(seed):
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(seed)
    d, dtype = r.choice([64, 128]), r.choice(["bf16", "fp16"])
    page, Hkv, G = r.choice([16, 32, 64, 128, 256]), r.choice([1, 2, 3]), r.choice([1, 2, 3, 5, 8, 17])
    B, T = r.choice([1, 2, 5, 20]), r.choice([1, 2, 5, 11, 30, 64, 100])
    if B * T * G > 4000:
        B = 1
    longest = r.choice([5, 100, 400, 3000])
    new = [r.choice([T, T, r.randint(0, T)]) for _ in range(B)]
    ctx = [r.randint(0, longest) for _ in range(B)]
    window = r.choice([-1, -1, -1, 0, r.randint(0, longest)])
    kind = r.choice([None, "random", "deep", "chain"])
    tail = r.choice([0, 0, 3, 300])
    c = draft_cache(ctx, new, page, Hkv, d, dtype, seed=seed, weights=True, capacity_tail=tail)
    q = (torch.randn((B, T, Hkv * G, d), generator=c.g) * r.choice([1.0, 4.0])).to(c.dtype).cuda()
    parents = kind and random_trees(c.g, B, T, kind)
    fa.device_error()
    bad = {}
    if r.random() < 0.3:
        for b in range(B):
            if sum((ctx[b], new[b])):
                bad[b] = r.randrange(-(-(ctx[b] + new[b]) // page))
        kept = c.table.clone()
        for b, x in bad.items():
            c.table[b, x] = r.choice([-1, c.num_pages, 1 << 30])
    out = torch.full_like(q, float("nan"))
    lse = torch.full((B, Hkv * G, T), float("nan"), device="cuda")
    ragged = int32(new) if r.random() < 0.7 or any(n != T for n in new) else None
    got = fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, parents=kind and parents.cuda(),
                                  new_lens=ragged, window_left=window, out=out, lse=lse)
    assert fa.device_error() in ((0, FA_ERR_PAGE) if bad else (0,))
    drop = (lambda b, t: bad.get(b) == t // page) if bad else None
    check_tree(*got, tree_ref(c, q, default_scale(d), parents, new, window, drop=drop), seed)
    if bad:
        c.table = kept
    if kind is None:
        return
    leaf = [r.randint(-1, n - 1) for n in new]
    ref = accept_ref(c, parents, leaf, T, new)
    path, lens = fa.paged_accept(c.k, c.v, c.table, c.seqlens, int32(leaf), parents.cuda(),
                                 new_lens=int32(new), weights=c.w)
    assert fa.device_error() == 0
    assert torch.equal(path.cpu(), ref[0]) and torch.equal(lens.cpu(), ref[1])
    assert same_bits(c.k, ref[2]) and same_bits(c.v, ref[3]) and same_bits(c.w, ref[4])


@pytest.mark.parametrize("B,T,Hq,ctx,d", [(3, 100, 4, 20, 128), (3, 100, 4, 20, 64), (400, 7, 2, 60, 64),
                                          (400, 7, 2, 200, 64), (3, 300, 4, 500, 128),
                                          (5, 9, 4, 100, 128), (5, 9, 4, 9000, 64)])
def test_padding(B, T, Hq, ctx, d):
    """Sequences with no drafted token, few and all of them, in every way that calls are carried out:
    every padded row is 0, with LSE -inf, and the workspace's contents do not matter."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(B * T)
    new = [r.choice([0, 0, 1, T // 2, T]) for _ in range(B)]
    new[0], new[1] = 0, T
    c = draft_cache([r.randint(0, ctx) for _ in range(B)], new, 16, 1, d, "bf16", seed=T)
    q = torch.randn((B, T, Hq, d), generator=c.g).to(c.dtype).cuda()
    parents = random_trees(c.g, B, T)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    need = fa.paged_tree_workspace_size(B, T, Hq, 1, d, 16, c.max_pages)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    o, lse = fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, parents=parents.cuda(),
                                     new_lens=int32(new), out=out, lse=lse, workspace=ws)
    check_tree(o, lse, tree_ref(c, q, default_scale(d), parents, new), (B, T))
    for b, n in enumerate(new):
        assert (o[b, n:] == 0).all() and torch.isneginf(lse[b, :, n:]).all()


@pytest.mark.parametrize("seed", range(12))
def test_books(seed):
    """Random forks and changes of lengths of a changing set of tables, in a pool that runs out now
    and then; at the end everything is given back."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(seed)
    page, width, pages = r.choice([16, 64]), r.choice([3, 40, 700]), r.choice([20, 300, 20000])
    pool = Pool(pages)
    r.shuffle(pool.free)
    dev = fa.PagePool(int32(pool.refs), int32(pool.stack()), int32([len(pool.free)]))
    B = r.choice([1, 4, 60])
    tables = [([[-1] * width for _ in range(B)], [0] * B)]
    devs = [int32(tables[0][0])]

    def check(what):
        assert dev.num_free.tolist() == [len(pool.free)], what
        assert dev.refs.tolist() == pool.refs, what
        assert dev.free_pages.tolist() == pool.stack(), what

    for step in range(10):
        i = r.randrange(len(tables))
        table, lens = tables[i]
        if r.random() < 0.4 and len(tables) < 4:
            source = [r.randint(-1, len(table) - 1) for _ in range(r.choice([1, 7, 50]))]
            out = fa.paged_fork(dev, devs[i], int32(lens), int32(source), page)
            want = pool.fork(table, lens, source, page)
            for x, y in zip(out, want):
                assert x.tolist() == y, step
            tables.append((want[0], [max(n, 0) for n in want[1]]))
            devs.append(out.block_table)
        else:
            later = [r.choice([0, n, r.randint(0, width * page)]) for n in lens]
            got = fa.paged_resize(dev, devs[i], int32(lens), int32(later), page)
            want = pool.resize(table, lens, later, page)
            assert got.tolist() == want and devs[i].tolist() == table, step
            tables[i] = (table, want)
        check(step)
    for (table, lens), d in zip(tables, devs):
        fa.paged_resize(dev, d, int32(lens), int32([0] * len(lens)), page)
        pool.resize(table, lens, [0] * len(lens), page)
        check("end")
    assert sorted(pool.free) == list(range(pages)) and fa.device_error() == 0


def test_line_is_the_kernels_path():
    """A leaf's path from the kernel is the one that its attention sees."""
    import io_aware_attention_fa2_gb300 as fa
    T = 200
    c = draft_cache([50], [T], 16, 1, 64, "bf16")
    parents = random_trees(c.g, 1, T)
    for leaf in (0, 57, T - 1):
        path, lens = fa.paged_accept(c.k.clone(), c.v.clone(), c.table, c.seqlens, int32([leaf]),
                                     parents.cuda())
        want = line(parents[0].tolist(), leaf)
        assert path[0].tolist() == want + [-1] * (T - len(want)) and lens.tolist() == [50 + len(want)]
