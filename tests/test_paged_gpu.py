"""The paged key-value cache on the GPU: append, decode, key weights and eviction against plain
float64 implementations (paged_util), at the lengths, page sizes, head groups and masks where
they can go wrong; bad block tables and lengths; streams, graphs and repeated calls; and a run of
all of them together."""
import math

import pytest
import torch

from paged_util import (DT, Cache, check_decode, decode_ref, default_scale, evict_ref,
                        key_weights_ref, same_bits)

pytestmark = pytest.mark.gpu
FA_ERR_PAGE = -13


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def decode(c, q, scale=None, **kw):
    import io_aware_attention_fa2_gb300 as fa
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=q.device)
    return fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, scale=scale, out=out, lse=lse, **kw)


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 1000]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d,dtype,Hq,Hkv", [(64, "fp16", 4, 4), (128, "bf16", 8, 2),
                                            (128, "fp16", 16, 1), (64, "bf16", 40, 2)])
@pytest.mark.parametrize("B,tokens,window", [(1, 2048, -1), (1, 2049, -1), (3, 64, -1),
                                             (4, 700, -1), (4, 90000, 1700), (18, 500, -1),
                                             (38, 256, -1), (60, 130, 40), (152, 200, -1),
                                             (153, 250, -1)])
def test_decode_short_and_long_tables(page, d, dtype, Hq, Hkv, B, tokens, window):
    """Both sides of the rule that gives a unit to a cluster: few and many units, tables up to
    and past its tiles, windows that make long tables short."""
    r = torch.Generator().manual_seed(B * tokens)
    lens = [tokens] + torch.randint(0, min(tokens, 5000) + 1, (B - 1,), generator=r).tolist()
    c = Cache(lens, page, Hkv, d, dtype, seed=tokens + page, weights=True)
    q = c.query(Hq)
    before = c.w.clone()
    o, lse = decode(c, q, window_left=window)
    assert same_bits(c.w, before)
    ref = decode_ref(c, q, default_scale(d), window)
    check_decode(c, q, o, lse, ref, (page, lens, window))
    o2, lse2 = decode(c, q, window_left=window, weights=c.w)
    check_decode(c, q, o2, lse2, ref, (page, lens, window, "weights"))
    check_weights(c, before, ref)


# ------------------------------------------------------------------------------------- decode
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
def test_decode_lengths(page, d, dtype):
    """Every length around the page and tile borders in one batch; rows behind the last token
    are NaN."""
    c = Cache(LENS, page, 2, d, dtype, seed=page + d)
    q = c.query(4)
    o, lse = decode(c, q)
    check_decode(c, q, o, lse, decode_ref(c, q, default_scale(d)), (page, d, dtype))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (12, 4), (16, 1), (20, 1), (34, 2),
                                    (64, 1), (70, 1), (130, 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_head_groups(Hq, Hkv, weights):
    c = Cache([130, 1, 517], 32, Hkv, 128, "bf16", seed=Hq, weights=weights)
    q = c.query(Hq)
    before = None if c.w is None else c.w.clone()
    o, lse = decode(c, q, weights=c.w)
    ref = decode_ref(c, q, default_scale(128))
    check_decode(c, q, o, lse, ref, (Hq, Hkv))
    if weights:
        check_weights(c, before, ref)


def check_weights(c, before, ref, lens=None):
    table, w0, w1 = c.table.cpu(), before.cpu(), c.w.cpu()
    touched = torch.zeros_like(w0, dtype=torch.bool)
    for b, n in enumerate(lens or c.lens):
        pg, row = c.rows(table, b, n)
        if n == 0:
            continue
        known = (pg >= 0) & (pg < c.num_pages)
        if not known.any():
            continue
        pg, row = pg[known], row[known]
        add, bound = ref[2][b].T[known], ref[5][b].T[known]
        got, want = w1[pg, :, row].double(), w0[pg, :, row].double() + add
        # the added value, and the sum's rounding to 32 bits (half a step)
        bad = (got - want).abs() - bound - want.abs() * 2.0 ** -24
        assert (bad <= 0).all(), float(bad.max())
        touched[pg, :, row] = True
    assert same_bits(w1[~touched], w0[~touched])


@pytest.mark.parametrize("n", [1, 64, 100, 2049, 5000])
@pytest.mark.parametrize("window", [0, 1, 15, 64, 100, 4096])
def test_decode_window(n, window):
    c = Cache([n, max(0, n - 40)], 16, 2, 64, "fp16", seed=n, weights=True)
    q = c.query(8)
    before = c.w.clone()
    o, lse = decode(c, q, window_left=window, weights=c.w)
    ref = decode_ref(c, q, default_scale(64), window)
    check_decode(c, q, o, lse, ref, (n, window))
    check_weights(c, before, ref)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_many_sequences(d):
    """More sequences than any block has threads, most of them empty or short."""
    lens = [(i * 37) % 90 if i % 3 else 0 for i in range(700)]
    c = Cache(lens, 16, 1, d, "bf16", seed=5)
    q = c.query(2)
    o, lse = decode(c, q)
    check_decode(c, q, o, lse, decode_ref(c, q, default_scale(d)), d)


@pytest.mark.parametrize("n", [9000, 40001])
def test_decode_long(n):
    c = Cache([n, 77], 64, 1, 128, "bf16", seed=n, weights=True)
    q = c.query(8)
    before = c.w.clone()
    o, lse = decode(c, q, weights=c.w)
    ref = decode_ref(c, q, default_scale(128))
    check_decode(c, q, o, lse, ref, n)
    check_weights(c, before, ref)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-6, 3.0])
def test_decode_scales(scale):
    """Scales of zero, of the other sign, and one whose softmax is almost one-hot."""
    c = Cache([300, 5], 32, 2, 64, "fp16", seed=8)
    q = c.query(4)
    o, lse = decode(c, q, scale=scale)
    check_decode(c, q, o, lse, decode_ref(c, q, scale), scale)


def test_decode_infinite_scores():
    """A key of -inf scores is never chosen; a sequence of them alone gives O = 0, LSE = -inf."""
    c = Cache([40, 20], 16, 1, 64, "bf16", seed=9)
    q = c.query(1).abs() + 0.5
    pg, row = c.rows(c.table, 0, 40)
    c.k[pg[3::4], row[3::4]] = -math.inf
    pg1, row1 = c.rows(c.table, 1, 20)
    c.k[pg1, row1] = -math.inf
    o, lse = decode(c, q)
    ref = decode_ref(c, q, default_scale(64), drop=lambda b, t: b == 1 or t % 4 == 3)
    check_decode(c, q, o, lse, ref, "inf")


def test_decode_lowest_values():
    """Keys at the type's lowest value give scores near the edge of fp32: still one-hot."""
    c = Cache([33], 16, 1, 64, "bf16", seed=10)
    q = c.query(1) * 0
    q[..., 0] = 1.0
    pg, row = c.rows(c.table, 0, 33)
    c.k[pg, row] = 0
    c.k[pg, row, :, 0] = torch.finfo(torch.bfloat16).min
    c.k[pg[7], row[7], :, 0] = 1.0
    o, lse = decode(c, q, scale=0.125)
    assert same_bits(o[0, 0], c.v[pg[7], row[7], 0])
    assert abs(float(lse[0, 0]) - 0.125) < 1e-6


def test_decode_shared_pages():
    """Two sequences read the same prefix pages; with weights both add to them."""
    c = Cache([96, 50], 32, 2, 64, "fp16", seed=11, weights=True)
    c.table[1, 0] = c.table[0, 0]
    c.table[1, 1] = c.table[0, 1]
    q = c.query(4)
    before = c.w.clone()
    o, lse = decode(c, q, weights=c.w)
    ref = decode_ref(c, q, default_scale(64))
    check_decode(c, q, o, lse, ref, "shared")
    pg, row = c.rows(c.table.cpu(), 0, 50)
    got = c.w.cpu()[pg, :, row].double()
    want = before.cpu()[pg, :, row].double() + ref[2][0].T[:50] + ref[2][1].T
    assert ((got - want).abs() <= ref[5][0].T[:50] + ref[5][1].T + 2.0 ** -23 * want.abs()).all()


def test_decode_bad_pages_are_left_out():
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([200, 200, 64], 16, 2, 128, "bf16", seed=12, weights=True)
    bad = {(0, 3): -1, (0, 12): c.num_pages, (1, 0): 2 ** 31 - 1, (1, 5): -2 ** 31}
    bad |= {(2, i): -1 for i in range(4)}
    for (b, i), value in bad.items():
        c.table[b, i] = value
    q = c.query(8)
    before = c.w.clone()
    o, lse = decode(c, q, weights=c.w)
    assert fa.device_error() == FA_ERR_PAGE
    ref = decode_ref(c, q, default_scale(128), drop=lambda b, t: (b, t // 16) in bad)
    check_decode(c, q, o, lse, ref, "bad pages")
    check_weights(c, before, ref)
    assert torch.isneginf(lse[2]).all() and (o[2] == 0).all()


def test_decode_bad_lengths():
    """A length beyond the table is the table's; a negative one is empty."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([64, 64, 10], 16, 1, 64, "bf16", seed=13)
    c.seqlens[:] = torch.tensor([65, 2 ** 31 - 1, -5], dtype=torch.int32)
    q = c.query(2)
    o, lse = decode(c, q)
    assert fa.device_error() == FA_ERR_PAGE
    check_decode(c, q, o, lse, decode_ref(c, q, default_scale(64), lens=[64, 64, 0]), "lengths")


def test_decode_same_bits_again_and_in_any_batch():
    """The same call gives the same bits; so does a capture's replay with other lengths."""
    c = Cache([3000, 17, 801], 32, 4, 128, "bf16", seed=14, weights=True)
    q = c.query(16)
    w0 = c.w.clone()
    o, lse = decode(c, q, weights=c.w)
    w1 = c.w.clone()
    c.w.copy_(w0)
    o2, lse2 = decode(c, q, weights=c.w)
    assert same_bits(o, o2) and same_bits(lse, lse2) and same_bits(w1, c.w)


@pytest.mark.parametrize("max_pages", [None, 150])
def test_decode_other_stream_and_graph(max_pages):
    """Captured on a side stream with a kept workspace, replayed for other lengths; two graphs
    that share the workspace run one after the other. (The shorter table needs none.)"""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([700, 300], 16, 2, 64, "fp16", seed=15, weights=True, max_pages=max_pages)
    q = c.query(8)
    ws = torch.empty(fa.paged_decode_workspace_size(2, 8, 2, 64, 16, c.max_pages, True),
                     dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(2, 8, device="cuda")) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = c.w.clone()
    o, lse = decode(c, q, weights=c.w, workspace=ws, stream=side)
    side.synchronize()
    check_decode(c, q, o, lse, decode_ref(c, q, default_scale(64)), "side stream")
    graphs = []
    for out, l in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, weights=c.w, workspace=ws,
                               out=out, lse=l)
        graphs.append(g)
    for lens in ([700, 300], [0, 299], [33, 1]):
        c.seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.w.copy_(before)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = decode_ref(c, q, default_scale(64), lens=lens)
        for out, l in outs:
            check_decode(c, q, out, l, ref, lens)
        twice = (ref[0], ref[1], [2 * x for x in ref[2]], *ref[3:5], [4 * x + 2.0 ** -24 for x in ref[5]])
        check_weights(c, before, twice, lens)


def test_decode_overlapping_streams():
    """Four calls at once on four streams, each as when alone."""
    cs = [Cache([2000 + 300 * i, 40], 32, 2, 128, "bf16", seed=20 + i) for i in range(4)]
    qs = [c.query(8) for c in cs]
    alone = [decode(c, q) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for c, q, s in zip(cs, qs, streams):
            with torch.cuda.stream(s):
                got.append(decode(c, q))
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(got, alone):
            assert same_bits(o, o1) and same_bits(l, l1)


def test_calls_from_several_threads():
    """Decodes, evictions and key weights of different sizes enqueued by four threads at once, each
    on its own stream, each as when alone."""
    import threading

    import io_aware_attention_fa2_gb300 as fa
    jobs = []
    for i in range(4):
        n = [300, 60000, 1500, 9000][i]
        c = Cache([n, n // 3], 64, 2, 64, "bf16", seed=40 + i, weights=True, spare=20)
        q = c.query(4)
        out = free_table(c, 128)
        p = torch.randn((1, 100 + 70 * i, 2, 64), generator=c.g).to(c.dtype).cuda()
        lse = torch.full((1, 2, p.shape[1]), 6.0, device="cuda")
        jobs.append((c, q, out, p, lse))

    def work(c, q, out, p, lse, stream=None):
        o, l = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, stream=stream)
        kept, lens = fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, out, 128, 16, stream=stream)
        w = fa.key_weights(p, p, lse, causal=True, stream=stream)
        return o, l, kept, lens, w

    alone = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[i] = work(*jobs[i], stream=stream)
            stream.synchronize()
        except Exception as e:   # reported below: an exception would end the thread alone
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert same_bits(x, y)


def test_streams_given_as_handles():
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([3000, 70], 32, 2, 64, "fp16", seed=50)
    q = c.query(4)
    want = decode(c, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (0, side, side.cuda_stream, torch.cuda.default_stream()):
        o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, stream=stream)
        torch.cuda.synchronize()
        assert same_bits(o, want[0]) and same_bits(lse, want[1])


def test_chain_behind_other_work():
    """Every call right behind work that writes what it reads: copies, fills, PyTorch kernels and
    other calls, in a stream, in a graph, and across streams. (The kernels may be launched before
    the work in front of them ends, and must wait for it.)"""
    import io_aware_attention_fa2_gb300 as fa
    n = 4000
    c = Cache([n, 900], 16, 2, 64, "bf16", seed=60, weights=True, spare=40)
    q = c.query(8)
    want = [decode(c, q), None]
    ref_w = c.w.clone()
    decode(c, q, weights=ref_w)
    out = free_table(c, 256)
    good = [x.clone() for x in (q, c.k, c.v, c.table, c.seqlens, c.w, out)]
    state = [x.clone() for x in good]
    gq, gk, gv, gt, gs, gw, go = state
    o, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    p = torch.randn((1, 500, 2, 64), generator=c.g).to(c.dtype).cuda()
    pl = torch.full((1, 2, 500), 7.0, device="cuda")
    want_pw = fa.key_weights(p, p, pl, causal=True)
    gp, gpl, pw = torch.empty_like(p), torch.empty_like(pl), torch.empty_like(want_pw)
    kept = torch.empty((2, 2, 256), dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def spoil():
        for x in (*state, gp, gpl):
            x.zero_()

    def restore(kind):
        for x, y in zip((*state, gp, gpl), (*good, p, pl)):
            if kind == "copy":
                x.copy_(y)                            # a copy node
            else:                                     # a kernel (on the bits: NaN stays as it is)
                kind_of = torch.int16 if x.element_size() == 2 else torch.int32
                torch.bitwise_or(y.view(kind_of), 0, out=x.view(kind_of))

    def calls():
        fa.fa_key_weights(gp, gp, gpl, pw, True, default_scale(64))
        fa.fa_paged_decode(gq, gk, gv, gt, gs, o, lse, default_scale(64), weights=gw)
        fa.fa_paged_evict(gk, gv, gw, gt, gs, go, kept, lens, 31)
        fa.fa_paged_decode(gq, gk, gv, go, lens, o2, lse2, default_scale(64))

    o2, lse2 = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    results = []
    for kind in ("copy", "kernel"):
        for how in ("stream", "graph", "streams"):
            spoil()
            big.zero_()
            torch.cuda.synchronize()
            if how == "graph":
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    big.zero_()
                    restore(kind)
                    calls()
                g.replay()
            elif how == "stream":
                big.zero_()
                restore(kind)
                calls()
            else:
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    big.zero_()
                    restore(kind)
                torch.cuda.current_stream().wait_stream(side)
                calls()
            torch.cuda.synchronize()
            assert same_bits(o, want[0][0]) and same_bits(lse, want[0][1]), (kind, how)
            assert same_bits(pw, want_pw), (kind, how)
            results.append([x.clone() for x in (kept, lens, o2, lse2, gk, gv, gw)])
    for r in results[1:]:
        for x, y in zip(r, results[0]):
            assert same_bits(x, y)
    assert results[0][1].tolist() == [256, 256]


def test_decode_pool_past_2_31_elements():
    """Pages whose rows lie past 2^31 elements and 2^32 bytes."""
    page, Hkv, d = 64, 8, 128
    num_pages = 36000                     # 2.36e9 elements in each pool
    n = 300
    k = torch.zeros((num_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = Cache([n], page, Hkv, d, "bf16", seed=16, spare=0)
    k[-5:], v[-5:] = small.k, small.v
    table = (small.table + (num_pages - 5)).to(torch.int32)
    import io_aware_attention_fa2_gb300 as fa
    q = small.query(8)
    o, lse = fa.paged_attention(q, k, v, table, small.seqlens)
    o1, lse1 = decode(small, q)
    assert same_bits(o, o1) and same_bits(lse, lse1)
    # append and evict on the same far rows
    w = torch.zeros((num_pages, Hkv, page), device="cuda")
    w[-5:] = torch.rand((5, Hkv, page), device="cuda")
    new = torch.randn((1, 1, Hkv, d), device="cuda").to(torch.bfloat16)
    seqlens = small.seqlens + 1
    fa.fa_paged_append(new, -new, k, v, table, seqlens, weights=w)
    pg, row = int(table[0, n // page]), n % page
    assert same_bits(k[pg, row], new[0, 0]) and same_bits(v[pg, row], -new[0, 0])
    out = torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2)
    kept, lens = fa.paged_evict(k, v, w, table, seqlens, out, 100, 10)
    for i in (0, 50, 99):
        t = int(kept[0, 3, i])
        assert same_bits(k[i // page, i % page, 3], k[int(table[0, t // page]), t % page, 3])
    assert int(lens[0]) == 100


# ------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("weights", ["no", "zero", "given"])
@pytest.mark.parametrize("d,Hkv,dtype", [(64, 1, "fp16"), (128, 3, "bf16")])
def test_append(page, weights, d, Hkv, dtype):
    """Padded new tokens to their places; every other row keeps its bits."""
    import io_aware_attention_fa2_gb300 as fa
    lens = [5, 100, 16, 300, 7]
    new = [5, 37, 0, 1, 7]
    c = Cache(lens, page, Hkv, d, dtype, seed=page, weights=weights != "no")
    N = max(new)
    k, v = (torch.randn((5, N, Hkv, d), generator=c.g).to(DT[dtype]).cuda() for _ in range(2))
    w = torch.rand((5, Hkv, N), generator=c.g).cuda() if weights == "given" else None
    want = [c.k.clone(), c.v.clone(), None if c.w is None else c.w.clone()]
    for b in range(5):
        pg, row = c.rows(c.table, b, lens[b])
        s = slice(lens[b] - new[b], lens[b])
        want[0][pg[s], row[s]], want[1][pg[s], row[s]] = k[b, :new[b]], v[b, :new[b]]
        if c.w is not None:
            want[2][pg[s], :, row[s]] = w[b, :, :new[b]].T if w is not None else 0.0
    fa.fa_paged_append(k, v, c.k, c.v, c.table, c.seqlens,
                       new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), w=w,
                       weights=c.w)
    for got, ref in zip((c.k, c.v, c.w), want):
        assert (got is None) == (ref is None) and (got is None or same_bits(got, ref))


def test_append_whole_prompt_without_lengths():
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([130, 130], 64, 2, 128, "bf16", seed=3)
    k, v = (torch.randn((2, 130, 2, 128), generator=c.g).to(c.dtype).cuda() for _ in range(2))
    fa.fa_paged_append(k, v, c.k, c.v, c.table, c.seqlens)
    for b in range(2):
        pg, row = c.rows(c.table, b, 130)
        assert same_bits(c.k[pg, row], k[b]) and same_bits(c.v[pg, row], v[b])


def test_append_bad_places_are_dropped():
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([40, 40, 40], 16, 2, 64, "fp16", seed=4, weights=True)
    c.table[0, 2] = c.num_pages            # tokens 32..39 of sequence 0
    c.seqlens[1] = 3                       # tokens -5..-1 of sequence 1 do not exist
    c.seqlens[2] = 48 + 4                  # tokens 48..51 are behind the table
    k = torch.randn((3, 8, 2, 64), generator=c.g).to(c.dtype).cuda()
    want = [c.k.clone(), c.v.clone(), c.w.clone()]
    pg, row = c.rows(c.table, 1, 3)
    want[0][pg, row] = want[1][pg, row] = k[1, 5:]
    want[2][pg, :, row] = 0
    page2 = int(c.table[2, 2])
    want[0][page2, 12:] = want[1][page2, 12:] = k[2, :4]
    want[2][page2, :, 12:] = 0
    fa.fa_paged_append(k, k.clone(), c.k, c.v, c.table, c.seqlens, weights=c.w)
    assert fa.device_error() == FA_ERR_PAGE
    for got, ref in zip((c.k, c.v, c.w), want):
        assert same_bits(got, ref)


# -------------------------------------------------------------------------------- key weights
def prompt(B, N, Hq, Hkv, d, dtype, causal, window, lens, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, N, Hq, d), generator=g).to(DT[dtype])
    k = torch.randn((B, N, Hkv, d), generator=g).to(DT[dtype])
    scale = default_scale(d)
    i = torch.arange(N)
    lse = torch.empty((B, Hq, N), dtype=torch.float64)
    for b in range(B):
        see = (i[None] < (N if lens is None else lens[b])).expand(N, N).clone()
        if causal:
            see &= i[None] <= i[:, None]
        if window[0] >= 0:
            see &= i[None] >= i[:, None] - window[0]
        if window[1] >= 0:
            see &= i[None] <= i[:, None] + window[1]
        for h in range(Hq):
            s = q[b, :, h].double() @ k[b, :, h // (Hq // Hkv)].double().T * scale
            lse[b, h] = torch.logsumexp(s.masked_fill(~see, -math.inf), 1)
    return q.cuda(), k.cuda(), lse.float().cuda(), scale


def check_key_weights(B, N, Hq, Hkv, d, dtype, causal, window=(-1, -1), lens=None, poison=False):
    import io_aware_attention_fa2_gb300 as fa
    q, k, lse, scale = prompt(B, N, Hq, Hkv, d, dtype, causal, window, lens, N + d)
    if poison:   # padding holds NaN, and so does its LSE
        for b, n in enumerate(lens):
            q[b, n:] = k[b, n:] = float("nan")
            lse[b, :, n:] = float("nan")
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, Hkv, N), float("nan"), device="cuda")
    w = fa.key_weights(q, k, lse, causal=causal, window=window, seqlens_k=lens_t, out=out)
    ref, bound = key_weights_ref(q, k, lse, scale, causal, window, lens)
    w = w.double().cpu()
    assert torch.isfinite(w).all()
    assert ((w - ref).abs() <= bound).all(), float(((w - ref).abs() - bound).max())
    return w


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_key_weights_lengths(N, causal, d, dtype):
    w = check_key_weights(2, N, 2, 2, d, dtype, causal)
    # every query's probabilities sum to one: N of them for each head
    assert (w.sum(-1) - N).abs().max() < N * 2.0 ** -12


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (6, 2), (16, 1)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_key_weights_head_groups(Hq, Hkv, d, dtype):
    check_key_weights(2, 300, Hq, Hkv, d, dtype, True)


@pytest.mark.parametrize("window", [(0, -1), (40, -1), (500, -1), (-1, 0), (-1, 70), (30, 30),
                                    (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_key_weights_windows(window, causal):
    check_key_weights(1, 520, 2, 2, 64, "bf16", causal, window)


@pytest.mark.parametrize("lens", [[400, 1, 0, 129], [256, 128, 300, 399]])
@pytest.mark.parametrize("window", [(-1, -1), (60, -1)])
def test_key_weights_padding(lens, window):
    """NaN behind every sequence's end; an empty sequence; queries with no visible key."""
    check_key_weights(4, 400, 4, 2, 128, "bf16", True, window, lens, poison=True)
    check_key_weights(4, 400, 2, 2, 64, "fp16", False, window, lens, poison=True)


def test_key_weights_rows_without_keys():
    """A window that leaves queries nothing: their LSE is -inf and they add nothing."""
    import io_aware_attention_fa2_gb300 as fa
    q, k, lse, scale = prompt(1, 200, 2, 2, 64, "bf16", False, (-1, -1), None, 7)
    lse[0, 0, 50:120] = -math.inf
    w = fa.key_weights(q, k, lse)
    ref, bound = key_weights_ref(q, k, lse, scale)
    assert ((w.double().cpu() - ref).abs() <= bound).all()


def test_key_weights_same_bits_and_streams():
    import io_aware_attention_fa2_gb300 as fa
    q, k, lse, _ = prompt(2, 700, 8, 2, 128, "bf16", True, (-1, -1), None, 8)
    alone = fa.key_weights(q, k, lse, causal=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [fa.key_weights(q, k, lse, causal=True, stream=s) for s in streams]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = fa.key_weights(q, k, lse, causal=True)
    captured.zero_()
    g.replay()
    torch.cuda.synchronize()
    for w in (*got, captured):
        assert same_bits(w, alone)


# -------------------------------------------------------------------------------------- evict
def evict(c, out_table, budget, recent):
    import io_aware_attention_fa2_gb300 as fa
    return fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, out_table, budget, recent)


def check_evict(c, out_table, budget, recent):
    kept, lens, k, v, w = evict_ref(c, out_table, budget, recent)
    got = evict(c, out_table, budget, recent)
    assert torch.equal(got[0].cpu(), kept)
    assert torch.equal(got[1].cpu(), lens)
    assert same_bits(c.k, k) and same_bits(c.v, v) and same_bits(c.w, w)


def free_table(c, budget):
    """Pages of c's spare ones for every sequence."""
    n = -(-budget // c.page)
    return c.free[:n * len(c.lens)].view(len(c.lens), n).cuda().contiguous()


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 3), (100, 100), (100, 0),
                                           (257, 31), (1500, 200)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128)])
def test_evict(budget, recent, in_place, page, d):
    lens = [0, 1, budget, budget + 1, 2500, 777]
    spare = len(lens) * -(-budget // page)
    c = Cache(lens, page, 2, d, "bf16", seed=budget + page, weights=True, spare=spare,
              max_pages=-(-max(2500, budget + 1) // page))
    if in_place:
        # rows of a table that is long enough for the budget; its unused entries are not read
        out = c.table.clone()
    else:
        out = free_table(c, budget)
    check_evict(c, out, budget, recent)


@pytest.mark.parametrize("kind", ["ties", "zeros", "special", "negative"])
def test_evict_ties_and_special_weights(kind):
    """Equal weights go to the oldest; -0 equals 0; NaN is the smallest, then -inf."""
    c = Cache([900, 333], 32, 3, 64, "fp16", seed=6, weights=True, spare=24)
    g = c.g
    shape = c.w.shape
    if kind == "ties":
        w = torch.randint(0, 4, shape, generator=g).float()
    elif kind == "zeros":
        w = torch.where(torch.rand(shape, generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0))
    elif kind == "negative":
        w = torch.randn(shape, generator=g)
    else:
        pick = torch.tensor([math.nan, -math.inf, math.inf, 0.0, -0.0, 1e-45, 3e38, -1.0])
        w = pick[torch.randint(0, 8, shape, generator=g)]
    c.w = w.cuda()
    check_evict(c, free_table(c, 350), 350, 40)


@pytest.mark.parametrize("n,in_place,ties", [(49152, False, False), (49153, True, True),
                                             (70001, False, True), (70001, True, False),
                                             (395000, False, True)])
def test_evict_long(n, in_place, ties):
    """Around and past what one CTA, and a cluster of them, keep of the weights on chip."""
    c = Cache([n, 300], 256, 1, 64, "bf16", seed=7, weights=True, spare=44,
              max_pages=-(-n // 256))
    if ties:
        c.w = torch.randint(0, 9, c.w.shape, generator=c.g).float().cuda()
    check_evict(c, c.table.clone() if in_place else free_table(c, 5000), 5000, 1000)


@pytest.mark.parametrize("rest", [0, 1, 2, 3])
@pytest.mark.parametrize("n,budget", [(700, 300), (50000, 4000)])
def test_evict_lowest_weights(n, budget, rest):
    """Fewer weights than the budget that are not NaN: the oldest of the NaN ones fill it, for
    candidates that end anywhere in a group of four and with NaN behind them."""
    n += rest
    c = Cache([n, n - 1], 64, 2, 64, "bf16", seed=n, weights=True, spare=2 * (budget // 64 + 1))
    c.w = torch.where(torch.rand(c.w.shape, generator=c.g) < 0.002,
                      torch.rand(c.w.shape, generator=c.g), torch.tensor(math.nan)).cuda()
    check_evict(c, free_table(c, budget), budget, 16)
    c.w = torch.full_like(c.w, math.nan)
    c.w[c.table[0, (n - 17) // 64], :, (n - 17) % 64] = -math.inf    # the last candidate
    check_evict(c, c.table.clone(), budget, 16)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_tables(in_place):
    """Thousands of pages in both tables; a pool past the bits that pre-select page numbers."""
    n, budget = 120000, 70000
    c = Cache([n, 40], 16, 1, 64, "fp16", seed=12, weights=True, spare=70000,
              max_pages=n // 16)
    out = c.table.clone() if in_place else free_table(c, budget)
    check_evict(c, out, budget, 999)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_again_and_again(in_place):
    """Evictions on end, as a decoding loop makes them."""
    c = Cache([600, 411], 16, 2, 64, "bf16", seed=8, weights=True, spare=80)
    for budget in (400, 399, 128, 17):
        out = c.table.clone() if in_place else free_table(c, budget)
        check_evict(c, out, budget, 9)
        c.lens = [min(n, budget) for n in c.lens]
        c.seqlens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
        if not in_place:
            used = set(out.flatten().tolist())
            old = [x for x in c.table.flatten().tolist() if x >= 0]
            c.table = out
            c.free = torch.tensor([x for x in c.free.tolist() if x not in used] + old,
                                  dtype=torch.int32)


def test_evict_into_earlier_own_pages():
    """out_table may name the sequence's own pages at an earlier place, shifted back by one."""
    c = Cache([500], 16, 2, 64, "fp16", seed=9, weights=True, spare=2)
    out = torch.cat([c.free[:1].cuda(), c.table[0, :19]]).view(1, 20).contiguous()
    check_evict(c, out, 320, 50)


def test_evict_refuses_bad_sequences():
    """A bad page, a bad length, or a destination that later tokens still sit in: nothing of that
    sequence moves, and the others are evicted as ever."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([200] * 6, 16, 2, 64, "bf16", seed=10, weights=True, spare=60)
    out = free_table(c, 100)
    good = Cache([200] * 6, 16, 2, 64, "bf16", seed=10, weights=True, spare=60)
    kept, lens, k, v, w = evict_ref(good, out, 100, 20)
    bad = [1, 2, 3, 4]
    for b in bad:                            # what a refused sequence leaves behind
        pg = out[b].long().cpu()
        k[pg], v[pg], w[pg] = good.k.cpu()[pg], good.v.cpu()[pg], good.w.cpu()[pg]
        kept[b] = -1
    out = out.clone()
    c.table[1, 12] = -1
    out[2, 6] = c.num_pages
    c.seqlens[3] = 13 * 16 + 1
    out[4, 2] = c.table[4, 3]
    got, new_lens = evict(c, out, 100, 20)
    assert fa.device_error() == FA_ERR_PAGE
    assert torch.equal(got.cpu(), kept)
    assert new_lens.tolist() == [100, 200, 200, 13 * 16 + 1, 200, 100]
    assert same_bits(c.k, k) and same_bits(c.v, v) and same_bits(c.w, w)


def test_evict_graph():
    c = Cache([900, 350], 32, 2, 128, "bf16", seed=11, weights=True, spare=30)
    out = free_table(c, 300)
    ref = evict_ref(c, out, 300, 30)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, lens = evict(c, out, 300, 30)
    for _ in range(2):                      # into free pages: the same again
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept.cpu(), ref[0]) and torch.equal(lens.cpu(), ref[1])
        assert same_bits(c.k, ref[2]) and same_bits(c.v, ref[3]) and same_bits(c.w, ref[4])


# ----------------------------------------------------------------------------- all of it together
@pytest.mark.parametrize("d,dtype,page", [(128, "bf16", 16), (64, "fp16", 64)])
def test_prompt_decode_evict_decode(d, dtype, page):
    """A padded prompt's forward, its key weights and its pages; decoding steps; an eviction in
    place; more steps over what was kept. Every step against float64 on the cache as it is."""
    import io_aware_attention_fa2_gb300 as fa
    B, H, N = 2, 4, 333
    lens = [333, 150]
    budget, recent = 160, 40
    c = Cache([0, 0], page, H, d, dtype, seed=12, weights=True, max_pages=-(-(N + 16) // page),
              spare=2 * -(-(N + 16) // page))
    c.table = c.free[:2 * c.max_pages].view(2, -1).cuda().contiguous()
    q, k, v = (torch.randn((B, N, H, d), generator=c.g).to(c.dtype).cuda() for _ in range(3))
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward(q, k, v, causal=True, seqlens_k=lens_t)
    w = fa.key_weights(q, k, lse, causal=True, seqlens_k=lens_t)
    assert (w.sum(-1).cpu() - torch.tensor(lens)[:, None]).abs().max() < N * 2.0 ** -10
    fa.fa_paged_append(k, v, c.k, c.v, c.table, lens_t, new_lens=lens_t, w=w, weights=c.w)
    # the last prompt token's attention, computed from the pages
    last = torch.stack([q[b, lens[b] - 1] for b in range(B)]).contiguous()
    c.lens, c.seqlens = list(lens), lens_t.clone()
    o1, lse1 = decode(c, last)
    ref = decode_ref(c, last, default_scale(d))
    check_decode(c, last, o1, lse1, ref, "prompt")
    want = torch.stack([o[b, lens[b] - 1] for b in range(B)]).double().cpu()
    # both sides are within the bound of the exact value
    assert ((o1.double().cpu() - want).abs() <= 2 * ref[3]).all()

    def step():
        new = [torch.randn((B, 1, H, d), generator=c.g).to(c.dtype).cuda() for _ in range(2)]
        c.lens = [n + 1 for n in c.lens]
        c.seqlens += 1
        fa.fa_paged_append(*new, c.k, c.v, c.table, c.seqlens, weights=c.w)
        query = c.query(H)
        before = c.w.clone()
        got = decode(c, query, weights=c.w)
        ref = decode_ref(c, query, default_scale(d))
        check_decode(c, query, *got, ref, c.lens)
        check_weights(c, before, ref)

    for _ in range(3):
        step()
    ref = evict_ref(c, c.table, budget, recent)
    kept, c.seqlens = evict(c, c.table.clone(), budget, recent)
    assert torch.equal(kept.cpu(), ref[0]) and same_bits(c.k, ref[2]) and same_bits(c.w, ref[4])
    c.lens = ref[1].tolist()
    for _ in range(3):
        step()
