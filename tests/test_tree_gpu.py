"""Attention of drafted tokens on the GPU against the plain float64 implementation (draft_util), at
the lengths, page sizes, head groups, trees and masks where it can go wrong; bad tables, lengths and
parents; what hidden rows hold; streams, graphs and repeated calls."""
import math

import pytest
import torch

from draft_util import check_tree, draft_cache, line, random_trees, tree_ref
from paged_util import default_scale, same_bits

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


def run(c, q, parents=None, new=None, window=-1, scale=None, **kw):
    import io_aware_attention_fa2_gb300 as fa
    B, T, Hq, _ = q.shape
    out = torch.full_like(q, float("nan"))
    lse = torch.full((B, Hq, T), float("nan"), device=q.device)
    return fa.paged_tree_attention(
        q, c.k, c.v, c.table, c.seqlens, parents=None if parents is None else parents.cuda(),
        new_lens=None if new is None else int32(new), scale=scale, window_left=window, out=out,
        lse=lse, **kw)


def queries(c, B, T, Hq, scale=1.0):
    return (torch.randn((B, T, Hq, c.d), generator=c.g) * scale).to(c.dtype).cuda()


CTX = [0, 1, 15, 16, 17, 63, 64, 65, 120, 127, 128, 129, 250, 256, 1000]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("T,Hq,Hkv", [(7, 4, 2), (40, 4, 1), (9, 32, 1)])
def test_context_lengths(page, d, dtype, T, Hq, Hkv):
    """Every length around the page and tile borders in one batch; rows behind the last token
    are NaN. Rows for less than one tile, for two, and for more."""
    B = len(CTX)
    c = draft_cache(CTX, [T] * B, page, Hkv, d, dtype, seed=page + d)
    q, parents = queries(c, B, T, Hq), random_trees(c.g, B, T)
    check_tree(*run(c, q, parents), tree_ref(c, q, default_scale(d), parents), (page, d, dtype))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 16, 1), (2, 8, 8), (3, 15, 3), (4, 40, 1),
                                      (5, 64, 2), (16, 16, 4), (31, 4, 1), (32, 4, 1), (33, 4, 1),
                                      (64, 4, 1), (65, 4, 1), (100, 3, 1), (130, 6, 1),
                                      (256, 4, 2), (257, 1, 1)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("kind", ["random", "deep", None])
def test_tokens_and_head_groups(T, Hq, Hkv, d, dtype, kind):
    ctx = [300, 0, 129]
    c = draft_cache(ctx, [T] * 3, 32, Hkv, d, dtype, seed=T * Hq)
    q = queries(c, 3, T, Hq)
    parents = kind and random_trees(c.g, 3, T, kind)
    check_tree(*run(c, q, parents), tree_ref(c, q, default_scale(d), parents), (T, Hq, kind))


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("B,tokens,T,Hq,Hkv,window", [
    (1, 4096, 8, 4, 1, -1), (1, 4097, 8, 4, 1, -1), (5, 3000, 3, 12, 3, -1), (4, 2048, 16, 32, 4, -1),
    (4, 2049, 16, 32, 4, -1), (9, 1024, 4, 16, 4, 300), (38, 1024, 2, 4, 2, -1), (38, 1025, 2, 4, 2, -1),
    (77, 512, 5, 3, 1, -1), (77, 513, 5, 3, 1, 100), (152, 400, 1, 8, 2, -1), (153, 400, 1, 8, 2, -1),
    (305, 128, 30, 4, 1, -1)])
def test_short_and_long_tables(d, dtype, B, tokens, T, Hq, Hkv, window):
    """Both sides of the rule that gives a unit to a cluster: few and many units, tables up to and
    past its tiles, sequences that leave some CTAs of a cluster without any."""
    r = torch.Generator().manual_seed(B * tokens)
    total = [tokens] + torch.randint(T, min(tokens, 2500) + 1, (B - 1,), generator=r).tolist()
    new = [T] + torch.randint(0, T + 1, (B - 1,), generator=r).tolist()
    c = draft_cache([n - m for n, m in zip(total, new)], new, 16, Hkv, d, dtype, seed=B)
    q, parents = queries(c, B, T, Hq), random_trees(c.g, B, T)
    got = run(c, q, parents, new, window)
    check_tree(*got, tree_ref(c, q, default_scale(d), parents, new, window), (B, tokens))
    again = run(c, q, parents, new, window)
    assert same_bits(got[0], again[0]) and same_bits(got[1], again[1])


def test_most_tokens():
    """1024 drafted tokens, as a chain without parents, as the same chain with them, and as trees."""
    T = 1024
    c = draft_cache([130, 5], [T, T], 64, 1, 64, "bf16", seed=3)
    q = queries(c, 2, T, 2)
    for kind in (None, "chain", "random"):
        parents = kind and random_trees(c.g, 2, T, kind)
        got = run(c, q, parents)
        check_tree(*got, tree_ref(c, q, default_scale(64), parents), kind)
        if kind == "chain":
            assert same_bits(got[0], chain[0]) and same_bits(got[1], chain[1])
        chain = got


@pytest.mark.parametrize("window", [0, 1, 2, 7, 64, 127, 128, 300, 5000])
@pytest.mark.parametrize("T,Hq,Hkv,kind", [(6, 4, 2, "random"), (70, 4, 1, "deep"),
                                           (40, 2, 2, None), (300, 2, 1, "deep")])
def test_window(window, T, Hq, Hkv, kind):
    ctx = [1000, 0, 64, 401]
    c = draft_cache(ctx, [T] * 4, 16, Hkv, 64, "fp16", seed=window)
    q = queries(c, 4, T, Hq)
    parents = kind and random_trees(c.g, 4, T, kind)
    check_tree(*run(c, q, parents, window=window),
               tree_ref(c, q, default_scale(64), parents, window=window), (window, T, kind))


@pytest.mark.parametrize("T,Hq,Hkv,d", [(6, 4, 2, 128), (50, 8, 2, 64), (150, 4, 1, 128)])
@pytest.mark.parametrize("window", [-1, 30])
def test_ragged_drafts(T, Hq, Hkv, d, window):
    """Fewer drafted tokens than the batch is wide, none, more (clamped); what the padding's queries
    and parents hold does not matter."""
    new = [T, 0, 1, T // 2, T + 9, T - 1, -3]
    real = [min(max(n, 0), T) for n in new]
    ctx = [200, 130, 0, 77, 128, 1, 0]
    c = draft_cache(ctx, real, 16, Hkv, d, "bf16", seed=T)
    q, parents = queries(c, 7, T, Hq), random_trees(c.g, 7, T, "deep")
    for b, n in enumerate(real):
        q[b, n:] = float("nan")
        parents[b, n:] = 1 << 30
    o, lse = run(c, q, parents, new, window)
    check_tree(o, lse, tree_ref(c, q, default_scale(d), parents, new, window), (T, window))
    for b, n in enumerate(real):
        assert (o[b, n:] == 0).all() and torch.isneginf(lse[b, :, n:]).all()


def test_many_sequences():
    """More sequences than any block has threads, most of them short."""
    ctx = [(i * 37) % 90 if i % 3 else 0 for i in range(700)]
    new = [i % 4 for i in range(700)]
    c = draft_cache(ctx, new, 16, 1, 64, "bf16", seed=5)
    q, parents = queries(c, 700, 3, 2), random_trees(c.g, 700, 3)
    check_tree(*run(c, q, parents, new), tree_ref(c, q, default_scale(64), parents, new), "many")


@pytest.mark.parametrize("n,T,Hq,d,dtype", [(40001, 4, 8, 128, "bf16"), (20000, 64, 4, 128, "fp16"),
                                            (33333, 17, 8, 64, "fp16")])
def test_long_contexts(n, T, Hq, d, dtype):
    """Sequences that many blocks share, beside short ones."""
    c = draft_cache([n, 77, 3000], [T] * 3, 64, 1, d, dtype, seed=n)
    q, parents = queries(c, 3, T, Hq, 2.0), random_trees(c.g, 3, T)
    check_tree(*run(c, q, parents), tree_ref(c, q, default_scale(d), parents), n)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-6, 3.0])
@pytest.mark.parametrize("T,Hq", [(5, 4), (80, 4)])
def test_scales(scale, T, Hq):
    """Scales of zero, of the other sign, and one whose softmax is almost one-hot."""
    c = draft_cache([900, 300], [T] * 2, 32, 1, 64, "bf16", seed=9)
    q, parents = queries(c, 2, T, Hq), random_trees(c.g, 2, T)
    check_tree(*run(c, q, parents, scale=scale),
               tree_ref(c, q, float(torch.tensor(scale, dtype=torch.float32)), parents), scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [6, 70])
def test_heavy_token_before_many_light_ones(dtype, T):
    """One token far above the others, early and late: what the others add to LSE and O is kept as
    far as the type can hold it, and a maximum that grows late rescales what came before."""
    for at in (3, 1990):
        c = draft_cache([2000], [T], 16, 1, 64, dtype, seed=at)
        q = queries(c, 1, T, 2)
        pg, row = c.rows(c.table.cpu(), 0, 2000)
        q[..., 0] = 4.0
        c.k[:, :, 0, 0] = 0.0
        c.k[pg[at], row[at], 0, 0] = 24.0     # scores 12 above, in units of e
        check_tree(*run(c, q), tree_ref(c, q, default_scale(64)), (dtype, at))


def plant(c, b, t, k=None, v=None):
    pg, row = int(c.table[b, t // c.page]), t % c.page
    if k is not None:
        c.k[pg, row] = k
    if v is not None:
        c.v[pg, row] = v


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("T,Hq", [(8, 2), (90, 2), (200, 3)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_values_do_not_matter(d, dtype, T, Hq, bad):
    """NaN and infinities in drafted tokens that a token does not see."""
    base = 140
    c = draft_cache([base], [T], 16, 1, d, dtype, seed=T)
    q = queries(c, 1, T, Hq)
    parents = random_trees(c.g, 1, T, "random")
    spoiled = [2, T // 2, T - 3]
    on_path = [i for i in range(T) if any(s in line(parents[0].tolist(), i) for s in spoiled)]
    clean = [i for i in range(T) if i not in on_path]
    assert len(clean) > T // 8 and len(on_path) >= len(spoiled)
    ref = tree_ref(c, q, default_scale(d), parents)
    for s in spoiled:
        plant(c, 0, base + s, bad, bad)
    o, lse = run(c, q, parents)
    pick = tuple(x[:, clean] for x in (o, ref[0], ref[2])) + tuple(
        x[:, :, clean] for x in (lse, ref[1], ref[3]))
    check_tree(pick[0], pick[3], (pick[1], pick[4], pick[2], pick[5]), (T, bad))


@pytest.mark.parametrize("T,Hq", [(4, 2), (70, 4)])
def test_values_behind_a_window_do_not_matter(T, Hq):
    """Tokens that fall out of the window one by one hold NaN."""
    base, window = 500, 200
    c = draft_cache([base], [T], 16, 1, 64, "bf16", seed=T)
    q = queries(c, 1, T, Hq)
    ref = tree_ref(c, q, default_scale(64), None, None, window)
    # token i sees base + i - 200 on: all of it is hidden from the last one
    first = base + T - 1 - window
    for t in range(0, first):
        plant(c, 0, t, float("nan"), float("nan"))
    o, lse = run(c, q, window=window)
    check_tree(o[:, -1:], lse[:, :, -1:], (ref[0][:, -1:], ref[1][:, :, -1:], ref[2][:, -1:],
                                           ref[3][:, :, -1:]), T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("where", [20, 205, 302])
@pytest.mark.parametrize("T,Hq", [(5, 4), (70, 4)])
def test_infinite_values_that_are_seen(dtype, where, T, Hq):
    """An infinity in V makes its column infinite, both signs or a NaN make it NaN, for the tokens
    that see it; in the context and among the drafted ones."""
    base, inf = 300, float("inf")
    c = draft_cache([base], [T], 64, 1, 64, dtype, seed=where)
    q = queries(c, 1, T, Hq)
    parents = torch.full((1, T), -1, dtype=torch.int32)
    parents[0, 3] = 2
    ref = tree_ref(c, q, default_scale(64), parents)
    pg, row = int(c.table[0, where // 64]), where % 64
    other = int(c.table[0, 10 // 64]), 10
    c.v[pg, row, 0, 1], c.v[pg, row, 0, 2], c.v[pg, row, 0, 3] = inf, -inf, float("nan")
    c.v[pg, row, 0, 4], c.v[other[0], other[1], 0, 4] = inf, -inf
    o, lse = (x.double().cpu() for x in run(c, q, parents))
    see = [i for i in range(T) if where < base or where - base in line(parents[0].tolist(), i)]
    hid = [i for i in range(T) if i not in see]
    assert (o[0, see, :, 1] == inf).all() and (o[0, see, :, 2] == -inf).all()
    assert torch.isnan(o[0, see][..., 3:5]).all()
    assert (o[0, hid, :, 4] == -inf).all()
    rest = [x for x in range(64) if x not in (1, 2, 3, 4)]
    assert ((o[0, :, :, rest] - ref[0][0, :, :, rest]).abs() <= ref[2][0, :, :, rest]).all()
    assert ((o[0, hid][..., 1:4] - ref[0][0, hid][..., 1:4]).abs() <= ref[2][0, hid][..., 1:4]).all()
    assert ((lse - ref[1]).abs() <= ref[3]).all()


# --------------------------------------------------------------------- what is checked on the GPU
@pytest.mark.parametrize("T,Hq", [(5, 4), (70, 4)])
@pytest.mark.parametrize("entry", [-1, -7, 10 ** 6, "num_pages"])
def test_bad_pages_are_left_out(T, Hq, entry):
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([200, 90], [T, T], 16, 2, 64, "bf16", seed=T)
    q, parents = queries(c, 2, T, Hq), random_trees(c.g, 2, T)
    c.table[0, 4] = c.num_pages if entry == "num_pages" else entry
    c.table[1, 90 // 16 + 1] = -1
    drop = lambda b, t: t // 16 == (4 if b == 0 else 90 // 16 + 1)   # noqa: E731
    o, lse = run(c, q, parents)
    assert fa.device_error() == FA_ERR_PAGE
    check_tree(o, lse, tree_ref(c, q, default_scale(64), parents, drop=drop), (T, entry))


def test_a_token_that_sees_nothing():
    """Its own page is bad and there is no context: O = 0 and LSE = -inf."""
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([0], [5], 16, 1, 64, "fp16")
    c.table[0, 0] = -1
    o, lse = run(c, queries(c, 1, 5, 4), random_trees(c.g, 1, 5))
    assert fa.device_error() == FA_ERR_PAGE
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T", [6, 80])
def test_bad_lengths_see_nothing(T):
    import io_aware_attention_fa2_gb300 as fa
    ctx = [100, 40, 7, 30]
    c = draft_cache(ctx, [T] * 4, 16, 1, 64, "bf16", seed=2)
    q = queries(c, 4, T, 4)
    lens = list(c.lens)
    lens[0], lens[1], lens[2] = -1, c.max_pages * 16 + 1, T - 1
    c.seqlens = int32(lens)
    o, lse = run(c, q)
    assert fa.device_error() == FA_ERR_PAGE
    assert (o[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    check_tree(o, lse, tree_ref(c, q, default_scale(64), lens=lens), "lengths")


@pytest.mark.parametrize("T", [6, 80])
def test_bad_parents_count_as_the_context(T):
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([100], [T], 16, 1, 64, "bf16", seed=2)
    q, parents = queries(c, 1, T, 4), random_trees(c.g, 1, T, "chain")
    for i, x in ((2, 2), (3, 10 ** 9), (4, -2), (5, 70)):
        parents[0, i] = x
    got = run(c, q, parents)
    assert fa.device_error() == FA_ERR_PAGE
    check_tree(*got, tree_ref(c, q, default_scale(64), parents), "parents")


def test_entries_behind_the_last_page_are_not_read():
    c = draft_cache([20, 500], [4, 4], 16, 1, 64, "bf16")
    c.table[0, 2:] = 10 ** 9
    q = queries(c, 2, 4, 2)
    check_tree(*run(c, q), tree_ref(c, q, default_scale(64)), "behind")


def test_refusals_of_the_binding():
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([20], [4], 16, 1, 64, "bf16")
    q, parents = queries(c, 1, 4, 2), random_trees(c.g, 1, 4).cuda()
    call = lambda **kw: fa.paged_tree_attention(   # noqa: E731
        **{**dict(q=q, k_pages=c.k, v_pages=c.v, block_table=c.table, seqlens=c.seqlens,
                  parents=parents), **kw})
    for name, bad in (("q", q[0]), ("q", q.float()), ("q", q.transpose(1, 2)),
                      ("parents", parents.long()), ("parents", parents[:, :3]),
                      ("new_lens", c.seqlens.cpu()), ("^o must", q[:, :2]), ("lse", q),
                      ("v_pages", c.v[1:]), ("workspace", torch.empty(8))):
        with pytest.raises(ValueError, match=name):
            call(**{"out" if "must" in name else name: bad})
    with pytest.raises(fa.FaError):
        call(scale=float("inf"))
    with pytest.raises(fa.FaError):
        call(out=q)


# ------------------------------------------------------------------- streams, graphs, repetition
@pytest.mark.parametrize("T,Hq", [(6, 4), (70, 8)])
def test_same_bits_every_time_and_on_other_streams(T, Hq):
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([5000, 300, 0], [T] * 3, 16, 2, 128, "bf16", seed=T)
    q, parents = queries(c, 3, T, Hq), random_trees(c.g, 3, T)
    first = run(c, q, parents)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        o, lse = run(c, q, parents, stream=stream if i % 2 else None)
        stream.synchronize()
        torch.cuda.synchronize()
        assert same_bits(o, first[0]) and same_bits(lse, first[1])
    need = fa.paged_tree_workspace_size(3, T, Hq, 2, 128, 16, c.max_pages)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")   # NaN as floats
    o, lse = run(c, q, parents, workspace=ws)
    assert same_bits(o, first[0]) and same_bits(lse, first[1])
    if need:
        with pytest.raises(fa.FaError):
            run(c, q, parents, workspace=ws[:need - 16])


@pytest.mark.parametrize("ctx", [3000, 6000])
def test_two_captured_graphs_and_an_eager_call(ctx):
    """Two graphs, each with a workspace of its own, replayed beside one another and beside eager
    calls, on lengths and trees that change between the replays; by one launch and by two."""
    T, Hq = 12, 8
    caches, graphs = [], []
    for s in (1, 2):
        c = draft_cache([ctx, 100], [T] * 2, 16, 2, 128, "bf16", seed=s)
        q, parents = queries(c, 2, T, Hq), random_trees(c.g, 2, T).cuda()
        run(c, q, parents)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(c, q, parents)
        caches.append((c, q, parents, out))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for step in range(4):
        for c, _, parents, _ in caches:
            c.lens = [c.lens[0] - 17 * step, c.lens[1] - 3 * step]
            c.seqlens.copy_(int32(c.lens))
            parents.copy_(random_trees(c.g, 2, T))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = [run(c, q, parents) for c, q, parents, _ in caches]
        torch.cuda.synchronize()
        for (c, q, parents, out), e in zip(caches, eager):
            check_tree(*out, tree_ref(c, q, default_scale(128), parents.cpu()), step)
            assert same_bits(out[0], e[0]) and same_bits(out[1], e[1])


def test_calls_from_several_threads():
    import threading
    cases = []
    for s in range(4):
        c = draft_cache([900 * s + 5, 60], [9] * 2, 16, 1, 64, "fp16", seed=s)
        q, parents = queries(c, 2, 9, 4), random_trees(c.g, 2, 9)
        cases.append((c, q, parents, run(c, q, parents)))
    torch.cuda.synchronize()
    failed = []

    def work(c, q, parents, want):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                o, lse = run(c, q, parents, stream=stream)
                torch.cuda.synchronize()
                assert same_bits(o, want[0]) and same_bits(lse, want[1])
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes (and 2^31 values) of keys, its last pages in use."""
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 40
    k, v = (torch.zeros((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    c = draft_cache([1500], [20], page, Hkv, d, "bf16", seed=1)
    high = torch.arange(pages - 1, pages - 1 - c.table.shape[1], -1, dtype=torch.int32,
                        device="cuda")
    k[high.long()], v[high.long()] = c.k[c.table[0].long()], c.v[c.table[0].long()]
    q, parents = queries(c, 1, 20, 16), random_trees(c.g, 1, 20)
    want = run(c, q, parents)
    c.k, c.v, c.table = k, v, high[None].contiguous()
    got = run(c, q, parents)
    assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    assert not math.isnan(float(got[1].sum()))


def test_one_drafted_token_is_a_decoding_step():
    """T = 1 beside paged_attention, within both kernels' bounds of the same reference."""
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([700, 15], [1, 1], 16, 2, 128, "bf16", seed=4)
    q = queries(c, 2, 1, 8)
    o, lse = run(c, q)
    ref = tree_ref(c, q, default_scale(128))
    check_tree(o, lse, ref, "tree")
    o1, lse1 = fa.paged_attention(q[:, 0].contiguous(), c.k, c.v, c.table, c.seqlens)
    check_tree(o1[:, None], lse1[:, :, None], ref, "decode")


def test_readme_example():
    """The README's block as it stands: its attention, and its sequences after the fork."""
    import os
    import re

    import io_aware_attention_fa2_gb300 as fa
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(path).read(), flags=re.S)
              if "paged_tree_attention" in b]
    assert len(blocks) == 1
    B, T, Hq, Hkv, d, page, width, num_pages = 3, 7, 4, 2, 64, 16, 12, 60
    lens, leaves, source = [50, 16, 0], [6, 3, -1], [0, 0, 2, 1]
    c = draft_cache(lens, [T] * B, page, Hkv, d, "bf16", seed=8)
    pool = fa.new_page_pool(num_pages)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    seqlens = fa.paged_resize(pool, table, int32([0] * B), int32(lens), page)
    k_pages = torch.full((num_pages, page, Hkv, d), float("nan"), dtype=c.dtype, device="cuda")
    v_pages = k_pages.clone()
    parents = torch.tensor([[-1, 0, 0, 1, 2, 3, 5]] * B, dtype=torch.int32)
    k, v = (torch.zeros((B, T, Hkv, d), dtype=c.dtype, device="cuda") for _ in "kv")
    rows = []
    for b, n in enumerate(lens):
        pg, row = c.rows(c.table, b, n + T)
        own = table[b].long().repeat_interleave(page)[:n]
        k_pages[own, row[:n]], v_pages[own, row[:n]] = c.k[pg[:n], row[:n]], c.v[pg[:n], row[:n]]
        k[b], v[b] = c.k[pg[n:], row[n:]], c.v[pg[n:], row[n:]]
        keep = list(range(n)) + [n + i for i in (line(parents[b].tolist(), leaves[b]))]
        rows.append((c.k[pg[keep], row[keep]], c.v[pg[keep], row[keep]]))
    q = queries(c, B, T, Hq)
    ns = dict(pool=pool, block_table=table, seqlens=seqlens, T=T, page_size=page, k=k, v=v, q=q,
              k_pages=k_pages, v_pages=v_pages, parents=parents.cuda(), source=int32(source),
              verify=lambda o: int32(leaves))
    exec(blocks[0], ns)
    check_tree(ns["o"], ns["lse"], tree_ref(c, q, default_scale(d), parents), "README")
    forked = ns["forked"]
    assert forked.seqlens.tolist() == [len(rows[s][0]) for s in source]
    for i, s in enumerate(source):
        n = len(rows[s][0])
        pg = forked.block_table[i].long().repeat_interleave(page)[:n]
        row = torch.arange(n, device="cuda") % page
        assert same_bits(k_pages[pg, row], rows[s][0]) and same_bits(v_pages[pg, row], rows[s][1])
