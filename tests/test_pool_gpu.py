"""Accept, copy, fork and resize on the GPU against plain implementations (draft_util): values bit
for bit, books entry for entry; bad entries; streams and graphs; and a step of speculative decoding
with branching sequences through all of the calls together."""
import random

import pytest
import torch

from draft_util import (Pool, accept_ref, check_tree, draft_cache, line, random_trees, tree_ref)
from paged_util import Cache, default_scale, same_bits

pytestmark = pytest.mark.gpu
FA_ERR_PAGE = -13


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------------------- accept
def check_accept(c, parents, leaf, T, new=None, **kw):
    import io_aware_attention_fa2_gb300 as fa
    ref = accept_ref(c, parents, leaf, T, new)
    lens = c.seqlens.clone()
    if parents is None:
        path, out = torch.empty((len(c.lens), T), dtype=torch.int32, device="cuda"), lens.clone()
        fa.fa_paged_accept(c.k, c.v, c.table, lens, int32(leaf), path, out, weights=c.w, **kw)
    else:
        path, out = fa.paged_accept(c.k, c.v, c.table, lens, int32(leaf), parents.cuda(),
                                    new_lens=None if new is None else int32(new), weights=c.w, **kw)
    torch.cuda.synchronize()
    assert torch.equal(path.cpu(), ref[0]) and torch.equal(out.cpu(), ref[1])
    assert same_bits(c.k, ref[2]) and same_bits(c.v, ref[3])
    assert c.w is None or same_bits(c.w, ref[4])
    assert same_bits(lens, c.seqlens)
    return ref


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d,dtype,Hkv", [(64, "fp16", 3), (128, "bf16", 2)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("T,kind", [(1, "random"), (7, "random"), (40, "deep"), (300, "deep")])
def test_accept(page, d, dtype, Hkv, weights, T, kind):
    """Contexts that end at and around a page's border; leaves from none to the last; the rest of
    the pools is left as it was."""
    ctx = [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 500]
    B = len(ctx)
    c = draft_cache(ctx, [T] * B, page, Hkv, d, dtype, seed=page + T, weights=weights)
    parents = random_trees(c.g, B, T, kind)
    leaf = torch.randint(-1, T, (B,), generator=c.g).tolist()
    leaf[0], leaf[-1] = T - 1, -1
    check_accept(c, parents, leaf, T)


@pytest.mark.parametrize("every", [1, 2, 3])
def test_accept_long_paths(every):
    """A path of up to 1024 tokens, more than one round: every row of it, or every second or third
    one, moves over rows that a later round still has to read."""
    T = 1024
    parents = torch.tensor([[i - every if i >= every else -1 for i in range(T)]] * 2,
                           dtype=torch.int32)
    for d in (64, 128):
        c = draft_cache([100, 7], [T, T], 16, 2, d, "bf16", seed=every, weights=True)
        check_accept(c, parents, [T - 1, T - 2], T)


def test_accept_chains_and_ragged_drafts():
    c = draft_cache([30, 5, 9], [6, 6, 6], 16, 1, 64, "bf16", weights=True)
    check_accept(c, None, [5, 2, -1], 6)
    new = [6, 0, 3, 6, 1]
    c = draft_cache([30, 5, 9, 0, 15], new, 16, 1, 64, "bf16", weights=True)
    parents = random_trees(c.g, 5, 6, "deep")
    for b, n in enumerate(new):
        parents[b, n:] = 10 ** 9
    check_accept(c, parents, [4, -1, 2, 5, 0], 6, new)


@pytest.mark.parametrize("what", ["length", "short", "leaf", "leaf_low", "parent", "source page",
                                  "target page"])
def test_accept_gives_up_a_bad_sequence(what):
    """Nothing of it moves; the others' tokens do."""
    import io_aware_attention_fa2_gb300 as fa
    T = 20
    c = draft_cache([15, 40], [T, T], 16, 2, 64, "bf16", weights=True, seed=3)
    parents = torch.tensor([[i - 3 if i > 2 else -1 for i in range(T)]] * 2, dtype=torch.int32)
    leaf = [19, 17]      # 1, 4, ... 19 of the first one: rows 16, 19, .. 34 to rows 15 .. 21
    before = [x.clone() for x in (c.k, c.v, c.w)]
    ref = accept_ref(c, parents, leaf, T)
    lens = c.seqlens.clone()
    table = c.table.clone()
    if what == "length":
        lens[0] = c.max_pages * 16 + 1
    elif what == "short":
        lens[0] = T - 1
    elif what == "leaf":
        leaf[0] = T
    elif what == "leaf_low":
        leaf[0] = -2
    elif what == "parent":
        parents[0, 7] = 8
    else:
        table[0, 2 if what == "source page" else 0] = c.num_pages
    path, out = fa.paged_accept(c.k, c.v, table, lens, int32(leaf), parents.cuda(), weights=c.w)
    assert fa.device_error() == FA_ERR_PAGE
    assert (path[0] == -1).all() and int(out[0]) == int(lens[0])
    assert torch.equal(path[1].cpu(), ref[0][1]) and int(out[1]) == int(ref[1][1])
    for got, old, want in zip((c.k, c.v, c.w), before, ref[2:]):
        first, second = c.table[0, :3].long(), c.table[1, :4].long()
        assert same_bits(got[first], old[first])
        assert same_bits(got[second], want[second.cpu()])


# ---------------------------------------------------------------------------------------- copy
@pytest.mark.parametrize("page,Hkv,d", [(16, 1, 64), (16, 8, 128), (32, 3, 64), (64, 8, 128),
                                        (128, 5, 128), (256, 2, 64)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("part", [False, True])
def test_copy(page, Hkv, d, weights, part):
    import io_aware_attention_fa2_gb300 as fa
    g = torch.Generator().manual_seed(page + Hkv)
    M = 37
    k, v = (torch.randn((2 * M + 3, page, Hkv, d), generator=g).bfloat16() for _ in "kv")
    k[5], v[6, :, 0] = float("nan"), float("inf")
    w = torch.randn((2 * M + 3, Hkv, page), generator=g) if weights else None
    order = torch.randperm(2 * M + 3, generator=g)
    src, dst = order[:M].clone(), order[M:2 * M].clone()
    src[:3] = src[3]                                      # a page to several others
    rows = torch.randint(0, page + 1, (M,), generator=g) if part else torch.full((M,), page)
    rows[0] = 0 if part else page
    dk, dv = k.cuda(), v.cuda()
    dw = None if w is None else w.cuda()
    skip_src, skip_dst = src.clone(), dst.clone()
    skip_src[7], skip_dst[7] = -1, -1
    fa.fa_paged_copy(dk, dv, skip_src.int().cuda(), skip_dst.int().cuda(),
                     rows=rows.int().cuda() if part else None, weights=dw)
    for m in range(M):
        if m == 7:
            continue
        n = int(rows[m])
        k[dst[m], :n], v[dst[m], :n] = k[src[m], :n], v[src[m], :n]
        if w is not None:
            w[dst[m], :, :n] = w[src[m], :, :n]
    assert same_bits(dk, k) and same_bits(dv, v) and (w is None or same_bits(dw, w))


def test_copy_leaves_bad_entries_out():
    import io_aware_attention_fa2_gb300 as fa
    k = torch.randn((8, 16, 1, 64), device="cuda").half()
    v = torch.randn_like(k)
    want = k.clone(), v.clone()
    want[0][7], want[1][7] = k[0], v[0]
    for bad in ((8, 1), (1, 8), (-1, 1), (1, -1), (-5, 2)):
        fa.fa_paged_copy(k, v, int32([bad[0], 0]), int32([bad[1], 7]))
        assert fa.device_error() == FA_ERR_PAGE
    for n in (-1, 17):
        fa.fa_paged_copy(k, v, int32([1, 0]), int32([2, 7]), rows=int32([n, 16]))
        assert fa.device_error() == FA_ERR_PAGE
    assert same_bits(k, want[0]) and same_bits(v, want[1])


def test_copy_beyond_32_bit_offsets():
    import io_aware_attention_fa2_gb300 as fa
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 8
    k, v = (torch.zeros((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k[pages - 1], v[pages - 1] = 3.0, 4.0
    fa.fa_paged_copy(k, v, int32([pages - 1, 0]), int32([pages - 3, pages - 2]))
    assert (k[pages - 3] == 3).all() and (v[pages - 3] == 4).all()
    assert float(k[:pages - 4].abs().max()) == 0 and float(k[pages - 2].abs().max()) == 0


# ------------------------------------------------------------------------------ fork and resize
def books(pool):
    import io_aware_attention_fa2_gb300 as fa
    return fa.PagePool(int32(pool.refs), int32(pool.stack()), int32([len(pool.free)]))


def check_books(got, pool, what=None):
    assert got.num_free.tolist() == [len(pool.free)], what
    assert got.refs.tolist() == pool.refs, what
    assert got.free_pages.tolist() == pool.stack(), what


def shuffled_pool(r, num_pages):
    pool = Pool(num_pages)
    r.shuffle(pool.free)
    return pool


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("B,longest", [(1, 100), (3, 5000), (40, 700), (1500, 40), (8192, 20)])
def test_resize_there_and_back(page, B, longest):
    """Growth, changes in both directions at once, and the end of every sequence."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(B + longest)
    width = -(-longest // page) + 1
    pool = shuffled_pool(r, B * width + 5)
    table = [[-1] * width for _ in range(B)]
    dev, dev_table = books(pool), int32(table)
    lens = [0] * B
    for step in range(5):
        later = [r.randint(0, longest) if r.random() < 0.8 else x for x in lens]
        if step == 4:
            later = [0] * B
        got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), page)
        assert got.tolist() == pool.resize(table, lens, later, page), step
        assert dev_table.tolist() == table, step
        check_books(dev, pool, step)
        lens = later
    assert len(pool.free) == B * width + 5


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("B,C,longest", [(1, 4, 100), (2, 3, 3000), (30, 70, 400), (5, 1300, 50),
                                         (64, 64, 40000)])
def test_fork_and_the_end_of_all(page, B, C, longest):
    """Sequences forked, the old ones ended, the new ones forked again and ended in two steps:
    pages that several tables give up in one call return once, by the last."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(B + C)
    width = -(-longest // page)
    lens = [r.choice([0, page, longest, r.randint(0, longest)]) for _ in range(B)]
    pool = shuffled_pool(r, sum(-(-n // page) for n in lens) + 2 * C + 3)
    table = [[-1] * width for _ in range(B)]
    pool.resize(table, [0] * B, lens, page)
    dev, tables = books(pool), [(int32(table), table, lens)]
    for _ in range(2):
        dev_old, old, old_lens = tables[-1]
        source = [r.randint(-1, len(old) - 1) for _ in range(C)]
        got = fa.paged_fork(dev, dev_old, int32(old_lens), int32(source), page)
        want = pool.fork(old, old_lens, source, page)
        for name, x, y in zip(got._fields, got, want):
            assert x.tolist() == y, name
        check_books(dev, pool)
        tables.append((got.block_table, want[0], want[1]))
    for i in (0, 2, 1):
        dev_table, table, lens = tables[i]
        half = [n // 2 if i == 2 else 0 for n in lens]
        for later in (half, [0] * len(lens)):
            got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), page)
            assert got.tolist() == pool.resize(table, lens, later, page)
            assert dev_table.tolist() == table
            check_books(dev, pool, (i, later[:4]))
            lens = later
    assert len(pool.free) == len(pool.refs) and not any(pool.refs)


@pytest.mark.parametrize("B,width,page,spare", [(64, 2100, 16, 5), (152, 900, 64, 5),
                                                (700, 200, 16, 5), (150, 1000, 16, -20000),
                                                (8192, 16, 256, 5)])
def test_large_tables(B, width, page, spare):
    """Tables that all SMs work on: growth, changes both ways, a pool that runs out, forks and the
    end of those that share pages, in one call."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(B)
    longest = width * page
    pool = shuffled_pool(r, B * width // 2 + spare)
    table = [[-1] * width for _ in range(B)]
    dev, dev_table = books(pool), int32(table)
    lens = [0] * B
    for step in range(3):
        later = [r.randint(0, longest // (2 if step else 3)) if r.random() < 0.9 else n for n in lens]
        later[r.randrange(B)] = longest
        got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), page)
        lens = pool.resize(table, lens, later, page)
        assert got.tolist() == lens, step
        assert dev_table.tolist() == table, step
        check_books(dev, pool, step)
    source = [r.randrange(B // 3) for _ in range(B)]   # several of the same sequence
    got = fa.paged_fork(dev, dev_table, int32(lens), int32(source), page)
    new, new_lens = pool.fork(table, lens, source, page)[:2]
    assert got.block_table.tolist() == new and got.seqlens.tolist() == new_lens
    check_books(dev, pool, "fork")
    new_lens = [max(n, 0) for n in new_lens]
    for t, dev_t, n, to in ((table, dev_table, lens, 0), (new, got.block_table, new_lens, page),
                            (new, got.block_table, [min(x, page) for x in new_lens], 0)):
        later = [min(x, to) for x in n]
        granted = fa.paged_resize(dev, dev_t, int32(n), int32(later), page)
        assert granted.tolist() == pool.resize(t, n, later, page) == later
        assert dev_t.tolist() == t
        check_books(dev, pool, to)
    assert len(pool.free) == len(pool.refs) and fa.device_error() == 0


@pytest.mark.parametrize("B,width,page", [(40, 5000, 16), (300, 500, 16)])
def test_few_pages_of_large_tables(B, width, page):
    """Steps of a few tokens, both ways, over tables that are large and mostly empty; children that
    give up the same few pages in one call."""
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(B)
    pool = shuffled_pool(r, 8 * B)
    table = [[-1] * width for _ in range(B)]
    dev, dev_table = books(pool), int32(table)
    lens = [0] * B
    for step in range(6):
        later = [max(0, n + r.randint(-20, 40)) for n in lens]
        got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), page)
        lens = pool.resize(table, lens, later, page)
        assert got.tolist() == lens and dev_table.tolist() == table, step
        check_books(dev, pool, step)
    source = [r.randrange(B // 4) for _ in range(B)]
    got = fa.paged_fork(dev, dev_table, int32(lens), int32(source), page)
    new, new_lens = pool.fork(table, lens, source, page)[:2]
    for dev_t, t, n in ((dev_table, table, lens), (got.block_table, new, new_lens)):
        fa.paged_resize(dev, dev_t, int32(n), int32([0] * B), page)
        pool.resize(t, n, [0] * B, page)
        assert dev_t.tolist() == t
        check_books(dev, pool, "end")
    assert len(pool.free) == 8 * B and fa.device_error() == 0


def test_large_tables_on_two_streams():
    """Two captured graphs, each with a pool of its own, replayed beside one another, and eager calls
    on a third pool meanwhile: the books of each as when it runs alone."""
    import io_aware_attention_fa2_gb300 as fa
    B, width, page = 160, 900, 16

    def work(seed):
        g = torch.Generator().manual_seed(seed)
        pool = fa.new_page_pool(B * width)
        pool.free_pages.copy_(torch.randperm(B * width, generator=g))
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        zero = int32([0] * B)
        lens = [torch.randint(0, width * page, (B,), generator=g, dtype=torch.int32).cuda()
                for _ in range(2)]
        source = torch.randint(0, B // 2, (B,), generator=g, dtype=torch.int32).cuda()

        def run():
            a = fa.paged_resize(pool, table, zero, lens[0], page)
            b = fa.paged_resize(pool, table, a, lens[1], page)
            child = fa.paged_fork(pool, table, b, source, page)
            kept = [x.clone() for x in (*pool, table, *child)]
            c = fa.paged_resize(pool, table, b, zero, page)
            fa.paged_resize(pool, child.block_table, child.seqlens.clamp(min=0), zero, page)
            return [*pool, table, a, b, c, *child, *kept]
        return run, pool

    def state(pool):
        return [x.clone() for x in pool]

    jobs = [work(s) for s in (1, 2, 3)]
    start = [state(pool) for _, pool in jobs]
    # alone, twice: the second run finds the stack as the first one left it
    alone = [[[x.clone() for x in run()] for _ in range(2)] for run, _ in jobs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for (run, _), s in zip(jobs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(run())
        graphs.append(graph)
    for (_, pool), books_ in zip(jobs, start):
        for x, y in zip(pool, books_):
            x.copy_(y)
    torch.cuda.synchronize()
    for step in range(2):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = jobs[2][0]()
        torch.cuda.synchronize()
        for got, want in zip((*outs, eager), alone):
            for i, (x, y) in enumerate(zip(got, want[step])):
                assert torch.equal(x, y), (step, i)
    assert fa.device_error() == 0


def test_large_tables_with_bad_entries():
    """Of 200 sequences one names a page outside the pool, one a free page, two the same page once
    referenced, and one has a length outside its table: recorded, the others are served."""
    import io_aware_attention_fa2_gb300 as fa
    B, width, page = 200, 700, 16
    pool = Pool(1000)
    table = [[-1] * width for _ in range(B)]
    lens = [64] * B
    pool.resize(table, [0] * B, lens, page)
    dev, dev_table = books(pool), int32(table)
    dev_table[3, 1], dev_table[7, 0] = 10 ** 6, pool.free[5]
    dev_table[50, 2] = table[90][3]
    lens[180] = width * page + 1
    later = [0] * 150 + [64] * 30 + [0] + [64] * 19
    got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), page)
    assert fa.device_error() == FA_ERR_PAGE
    assert got.tolist() == later[:180] + [lens[180]] + later[181:]
    assert (dev_table[:150] == -1).all() and dev_table[150:].tolist() == table[150:]
    # which of the two entries counted is not told: the page returned once
    back = {p for b in range(150) for p in table[b][:4]}
    back -= {table[3][1], table[7][0], table[50][2]}
    n = int(dev.num_free[0])
    assert n == len(pool.free) + len(back)
    assert dev.free_pages[:len(pool.free)].tolist() == pool.free
    assert set(dev.free_pages[len(pool.free):n].tolist()) == back
    assert all(dev.refs[p] == 0 for p in back)


def test_an_empty_pool():
    """What the pool cannot give is refused from there on; pages given back in the same call count;
    sequences that need none are served."""
    import io_aware_attention_fa2_gb300 as fa
    pool = Pool(10)
    table = [[-1] * 8 for _ in range(5)]
    lens = [64, 20, 0, 16, 10]
    pool.resize(table, [0] * 5, lens, 16)
    dev, dev_table = books(pool), int32(table)
    for later in ([64, 60, 100, 20, 10], [0, 60, 50, 10 ** 6, 16], [0, 200, 0, 16, 3]):
        later[3] = min(later[3], 128)
        got = fa.paged_resize(dev, dev_table, int32(lens), int32(later), 16)
        want = pool.resize(table, lens, later, 16)
        assert got.tolist() == want and dev_table.tolist() == table
        check_books(dev, pool)
        # (200 tokens are more than the table has columns for: refused for that, too)
        assert fa.device_error() == (FA_ERR_PAGE if max(later) > 128 else 0)
        lens = want
    got = fa.paged_fork(dev, dev_table, int32(lens), int32([1, 4, 3, -1, 4] * 4), 16)
    want = pool.fork(table, lens, [1, 4, 3, -1, 4] * 4, 16)
    assert -1 in want[1]
    for x, y in zip(got, want):
        assert x.tolist() == y
    check_books(dev, pool)
    assert fa.new_page_pool(3).free_pages.tolist() == [2, 1, 0]


def test_bad_books_are_recorded():
    """Entries outside the pool, pages that no table should hold, lengths outside the table."""
    import io_aware_attention_fa2_gb300 as fa
    pool = Pool(12)
    table = [[-1] * 4 for _ in range(3)]
    pool.resize(table, [0] * 3, [64, 40, 20], 16)
    dev, dev_table = books(pool), int32(table)
    # an entry outside the pool, and one of a free page, are not given back
    dev_table[0, 1], dev_table[0, 2] = 99, pool.free[0]
    got = fa.paged_resize(dev, dev_table, int32([64, 40, 20]), int32([0, 40, 20]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert got.tolist() == [0, 40, 20] and dev_table[0].tolist() == [-1] * 4
    assert dev.num_free.tolist() == [len(pool.free) + 2]
    assert dev.free_pages[:len(pool.free) + 2].tolist() == pool.free + [table[0][0], table[0][3]]
    refs = list(pool.refs)
    refs[table[0][0]] = refs[table[0][3]] = 0
    assert dev.refs.tolist() == refs
    # lengths
    for bad in (-1, 65):
        got = fa.paged_resize(dev, dev_table, int32([0, 40, bad]), int32([0, 40, 0]), 16)
        assert fa.device_error() == FA_ERR_PAGE and got.tolist() == [0, 40, bad]
        got = fa.paged_resize(dev, dev_table, int32([0, 40, 20]), int32([0, 40, bad]), 16)
        assert fa.device_error() == FA_ERR_PAGE and got.tolist() == [0, 40, 20]
    assert dev.refs.tolist() == refs
    # forks of bad sequences, and of one whose table has a bad entry
    out = fa.paged_fork(dev, dev_table, int32([0, 40, 65]), int32([3, -2, 2, -1]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert out.seqlens.tolist() == [-1, -1, -1, 0] and (out.block_table == -1).all()
    assert dev.refs.tolist() == refs
    dev_table[1, 0] = 12
    out = fa.paged_fork(dev, dev_table, int32([0, 32, 0]), int32([1]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert out.seqlens.tolist() == [32] and out.block_table[0, :2].tolist() == [-1, table[1][1]]
    # a count of free pages that the pool cannot have gives none
    for n in (-1, 13):
        broken = fa.PagePool(dev.refs.clone(), dev.free_pages.clone(), int32([n]))
        got = fa.paged_resize(broken, dev_table.clone(), int32([0, 40, 20]), int32([16, 40, 20]), 16)
        assert fa.device_error() == FA_ERR_PAGE and got.tolist() == [0, 40, 20]


def test_a_page_given_up_twice_returns_once():
    """One reference, but two tables that name the page."""
    import io_aware_attention_fa2_gb300 as fa
    dev = fa.new_page_pool(4)
    table = int32([[-1], [-1]])
    fa.paged_resize(dev, table, int32([0, 0]), int32([16, 16]), 16)
    table[1, 0] = table[0, 0]
    fa.paged_resize(dev, table, int32([16, 16]), int32([0, 0]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert dev.refs.tolist() == [0, 1, 0, 0] and dev.num_free.tolist() == [3]
    assert dev.free_pages.tolist() == [3, 2, 0, -1]


def test_refusals_of_the_binding():
    import io_aware_attention_fa2_gb300 as fa
    dev, table, lens = fa.new_page_pool(6), int32([[0, 1]]), int32([20])
    for bad, name in ((table.long(), "block_table"), (table[0], "block_table"),
                      (table.t(), "old_lens")):       # two sequences of one page
        with pytest.raises(ValueError, match=name):
            fa.paged_resize(dev, bad, lens, lens, 16)
    with pytest.raises(ValueError, match="refs"):
        fa.paged_resize(dev._replace(refs=dev.refs.float()), table, lens, lens, 16)
    with pytest.raises(ValueError, match="new_lens"):
        fa.paged_resize(dev, table, lens, lens.long(), 16)
    with pytest.raises(ValueError, match="source"):
        fa.paged_fork(dev, table, lens, table, 16)
    with pytest.raises(ValueError, match="page_size"):
        fa.paged_fork(dev, table, lens, lens, 2 ** 33)
    for page in (0, 24):
        with pytest.raises(fa.FaError):
            fa.paged_fork(dev, table, lens, int32([0]), page)
        with pytest.raises(fa.FaError):
            fa.paged_resize(dev, table, lens, lens.clone(), page)
    c = draft_cache([20], [4], 16, 1, 64, "bf16")
    with pytest.raises(ValueError, match="parents"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, int32([0]), int32([0]))
    with pytest.raises(ValueError, match="leaf"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, int32([0, 1]), int32([[-1, 0]]))
    with pytest.raises(ValueError, match="rows"):
        fa.fa_paged_copy(c.k, c.v, int32([0]), int32([1]), rows=int32([1, 2]))


# ---------------------------------------------------------------------------- all of them together
@pytest.mark.parametrize("captured", [False, True])
def test_speculation_and_branches(captured):
    """Steps of speculative decoding for a batch whose sequences are forked half way: room, append,
    tree attention, accept, and what was drafted in vain given back. Every step's attention and
    every sequence's tokens are compared with plain lists of tokens; at the end the pool is whole.
    Captured: a step is one graph, replayed with new contents of its inputs."""
    import io_aware_attention_fa2_gb300 as fa
    page, Hkv, Hq, d, T, B = 16, 2, 8, 64, 9, 3
    g, r = torch.Generator().manual_seed(11), random.Random(11)
    width, num_pages = 24, 160
    dev = fa.new_page_pool(num_pages)
    k_pages = torch.full((num_pages, page, Hkv, d), float("nan"), dtype=torch.bfloat16,
                         device="cuda")
    v_pages = k_pages.clone()
    weights = torch.full((num_pages, Hkv, page), float("nan"), device="cuda")

    def randn(*shape):
        return torch.randn(shape, generator=g).bfloat16()

    # prompts
    lens = [70, 16, 5]
    K = [randn(n, Hkv, d) for n in lens]
    V = [randn(n, Hkv, d) for n in lens]
    W = [torch.rand((n, Hkv), generator=g) for n in lens]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    seqlens = fa.paged_resize(dev, table, int32([0] * B), int32(lens), page)

    def padded(xs):
        return torch.nn.utils.rnn.pad_sequence(xs, batch_first=True).cuda()

    fa.fa_paged_append(padded(K), padded(V), k_pages, v_pages, table, seqlens, new_lens=seqlens,
                       w=padded(W).transpose(1, 2).contiguous(), weights=weights)

    def step(n, q, k, v, parents, leaf, table, seqlens):
        room = fa.paged_resize(dev, table, seqlens, seqlens + T, page)
        fa.fa_paged_append(k, v, k_pages, v_pages, table, room, weights=weights)
        o, lse = fa.paged_tree_attention(q, k_pages, v_pages, table, room, parents=parents)
        path, now = fa.paged_accept(k_pages, v_pages, table, room, leaf, parents, weights=weights)
        kept = fa.paged_resize(dev, table, room, now, page)
        seqlens.copy_(kept)
        return o, lse, path

    def sequences(table, seqlens):
        """Each sequence's tokens as they stand in the pages."""
        t, kp, vp, wp = (x.cpu() for x in (table, k_pages, v_pages, weights))
        out = []
        for b, n in enumerate(seqlens.tolist()):
            pg = t[b, :max(1, -(-n // page))].long().repeat_interleave(page)[:n]
            row = torch.arange(n) % page
            out.append((kp[pg, row], vp[pg, row], wp[pg, :, row]))
        return out

    def run_steps(count, table, seqlens):
        n = len(K)
        ins = [torch.empty((n, T, Hq, d), dtype=torch.bfloat16, device="cuda"),
               *(torch.empty((n, T, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"),
               torch.empty((n, T), dtype=torch.int32, device="cuda"),
               torch.empty((n,), dtype=torch.int32, device="cuda")]
        graph = None
        for _ in range(count):
            parents = random_trees(g, n, T, r.choice(["random", "deep"]))
            leaf = [r.randint(-1, T - 1) for _ in range(n)]
            fresh = [randn(n, T, Hq, d), randn(n, T, Hkv, d), randn(n, T, Hkv, d), parents,
                     torch.tensor(leaf, dtype=torch.int32)]
            for x, y in zip(ins, fresh):
                x.copy_(y)
            if not captured:
                o, lse, path = step(n, *ins, table, seqlens)
            else:
                if graph is None:
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        o, lse, path = step(n, *ins, table, seqlens)
                graph.replay()
            torch.cuda.synchronize()
            # the attention over a plain cache of the same tokens
            c = Cache([len(x) + T for x in K], page, Hkv, d, "bf16")
            for b in range(n):
                pg, row = c.rows(c.table, b, c.lens[b])
                c.k[pg, row] = torch.cat([K[b], fresh[1][b]]).cuda()
                c.v[pg, row] = torch.cat([V[b], fresh[2][b]]).cuda()
            check_tree(o, lse, tree_ref(c, fresh[0], default_scale(d), parents), "step")
            for b in range(n):
                keep = line(parents[b].tolist(), leaf[b])
                assert path[b].tolist() == keep + [-1] * (T - len(keep))
                K[b] = torch.cat([K[b], fresh[1][b, keep]])
                V[b] = torch.cat([V[b], fresh[2][b, keep]])
                W[b] = torch.cat([W[b], torch.zeros((len(keep), Hkv))])
            assert seqlens.tolist() == [len(x) for x in K]
            for b, (k, v, w) in enumerate(sequences(table, seqlens)):
                assert same_bits(k, K[b]) and same_bits(v, V[b]) and same_bits(w, W[b])

    run_steps(4, table, seqlens)
    # two continuations of the first sequence, one of the last, a new one; the others end
    source = [0, 2, 0, -1, 0]
    forked = fa.paged_fork(dev, table, seqlens, int32(source), page)
    fa.fa_paged_copy(k_pages, v_pages, forked.copy_src, forked.copy_dst, rows=forked.copy_rows,
                     weights=weights)
    fa.paged_resize(dev, table, seqlens, torch.zeros_like(seqlens), page)
    none = randn(0, Hkv, d), torch.zeros((0, Hkv))
    K = [none[0] if s < 0 else K[s] for s in source]
    V = [none[0] if s < 0 else V[s] for s in source]
    W = [none[1] if s < 0 else W[s] for s in source]
    table, seqlens = forked.block_table, forked.seqlens.clone()
    for b, (k, v, w) in enumerate(sequences(table, seqlens)):
        assert same_bits(k, K[b]) and same_bits(v, V[b]) and same_bits(w, W[b])
    run_steps(4, table, seqlens)
    fa.paged_resize(dev, table, seqlens, torch.zeros_like(seqlens), page)
    assert dev.num_free.tolist() == [num_pages] and not dev.refs.any()
    assert sorted(dev.free_pages.tolist()) == list(range(num_pages)) and (table == -1).all()
