"""Seeded random combinations of shape, type, page size, lengths, masks and options for the paged
cache's operators, each against its plain float64 implementation; what the binding and the library
refuse; and a serving step captured into a graph and replayed as its sequences grow."""
import math
import random

import pytest
import torch

from paged_util import (DT, Cache, check_decode, decode_ref, default_scale, evict_ref, same_bits)
from test_paged_gpu import check_evict, check_key_weights, check_weights, decode, free_table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def log_int(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


@pytest.mark.parametrize("seed", range(40))
def test_decode_fuzz(seed):
    r = random.Random(seed)
    d, dtype = r.choice([64, 128]), r.choice(["bf16", "fp16"])
    page = r.choice([16, 32, 64, 128, 256])
    Hkv, G = r.choice([1, 2, 3, 5, 8]), r.choice([1, 2, 3, 4, 7, 8, 16, 17, 24])
    if Hkv * G > 48:
        G = 1
    lens = [r.choice([0, log_int(r, 1, 3000), log_int(r, 1, 200)])
            for _ in range(r.choice([1, 2, 3, 9, 33]))]
    if sum(lens) * Hkv * G > 400000:
        lens = [n // 8 for n in lens]
    window = r.choice([-1, -1, 0, log_int(r, 1, 2000)])
    scale = r.choice([default_scale(d), default_scale(d), 0.5, -0.1])
    weights = r.random() < 0.5
    c = Cache(lens, page, Hkv, d, dtype, seed=seed, weights=weights,
              max_pages=max(1, -(-max(lens) // page)) + r.choice([0, 0, 1, 7]))
    q = c.query(Hkv * G, r.choice([0.1, 1.0, 3.0]))
    before = None if c.w is None else c.w.clone()
    o, lse = decode(c, q, scale=scale, window_left=window, weights=c.w)
    ref = decode_ref(c, q, scale, window)
    check_decode(c, q, o, lse, ref, (seed, lens, window, page, Hkv, G, d, dtype, scale))
    if weights:
        check_weights(c, before, ref)


@pytest.mark.parametrize("seed", range(25))
def test_key_weights_fuzz(seed):
    r = random.Random(1000 + seed)
    B, N = r.choice([1, 2, 3]), log_int(r, 1, 1500)
    Hkv, G = r.choice([1, 2, 3]), r.choice([1, 1, 2, 5])
    window = (r.choice([-1, -1, 0, log_int(r, 1, 900)]), r.choice([-1, -1, -1, log_int(r, 1, 900)]))
    lens = None if r.random() < 0.5 else [r.randint(0, N) for _ in range(B)]
    check_key_weights(B, N, Hkv * G, Hkv, r.choice([64, 128]), r.choice(["bf16", "fp16"]),
                      r.random() < 0.6, window, lens, poison=lens is not None)


@pytest.mark.parametrize("seed", range(25))
def test_evict_fuzz(seed):
    r = random.Random(2000 + seed)
    page, Hkv = r.choice([16, 32, 64, 256]), r.choice([1, 2, 5])
    lens = [r.choice([0, log_int(r, 1, 4000), log_int(r, 1, 300)])
            for _ in range(r.choice([1, 2, 6]))]
    budget = log_int(r, 1, max(2, max(lens)))
    c = Cache(lens, page, Hkv, r.choice([64, 128]), r.choice(["bf16", "fp16"]), seed=seed,
              weights=True, spare=len(lens) * -(-budget // page),
              max_pages=max(1, -(-max(max(lens), budget) // page)))
    if r.random() < 0.4:
        c.w = torch.randint(0, r.choice([2, 5, 50]), c.w.shape, generator=c.g).float().cuda()
    out = c.table.clone() if r.random() < 0.4 else free_table(c, budget)
    check_evict(c, out, budget, r.randint(0, budget))


@pytest.mark.parametrize("seed", range(20))
def test_append_fuzz(seed):
    import io_aware_attention_fa2_gb300 as fa
    r = random.Random(3000 + seed)
    B, Hkv, d = r.choice([1, 3, 20]), r.choice([1, 2, 7, 16]), r.choice([64, 128])
    dtype = r.choice(["bf16", "fp16"])
    N = r.choice([1, 1, log_int(r, 2, 300)])
    new = [r.randint(0, N) for _ in range(B)]
    lens = [n + r.choice([0, log_int(r, 1, 500)]) for n in new]
    weights = r.random() < 0.5
    c = Cache(lens, r.choice([16, 64, 256]), Hkv, d, dtype, seed=seed, weights=weights)
    k, v = (torch.randn((B, N, Hkv, d), generator=c.g).to(DT[dtype]).cuda() for _ in range(2))
    w = torch.rand((B, Hkv, N), generator=c.g).cuda() if weights and r.random() < 0.5 else None
    want = [c.k.clone(), c.v.clone(), None if c.w is None else c.w.clone()]
    for b in range(B):
        pg, row = c.rows(c.table, b, lens[b])
        pg, row = pg[lens[b] - new[b]:], row[lens[b] - new[b]:]
        want[0][pg, row], want[1][pg, row] = k[b, :new[b]], v[b, :new[b]]
        if weights:
            want[2][pg, :, row] = w[b, :, :new[b]].T if w is not None else 0.0
    fa.fa_paged_append(k, v, c.k, c.v, c.table, c.seqlens,
                       new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), w=w,
                       weights=c.w)
    for got, ref in zip((c.k, c.v, c.w), want):
        assert (got is None) == (ref is None) and (got is None or same_bits(got, ref))


def test_refusals_of_the_binding():
    """Wrong shapes, types, strides and devices are named before anything runs."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([40, 20], 16, 2, 64, "bf16", seed=1, weights=True)
    q = c.query(4)

    def refused(match, call, *args, **kw):
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)

    dec = fa.paged_attention
    refused("q must", dec, q[0], c.k, c.v, c.table, c.seqlens)
    refused("q must", dec, q.half(), c.k, c.v, c.table, c.seqlens)
    refused("q must", dec, q[:, ::2], c.k, c.v, c.table, c.seqlens)
    refused("v_pages", dec, q, c.k, c.v[:-1], c.table, c.seqlens)
    refused("k_pages", dec, q, c.k.transpose(1, 2), c.v, c.table, c.seqlens)
    refused("block_table", dec, q, c.k, c.v, c.table.long(), c.seqlens)
    refused("block_table", dec, q, c.k, c.v, c.table.cpu(), c.seqlens)
    refused("block_table", dec, q, c.k, c.v, c.table[:, :1], c.seqlens)
    refused("seqlens", dec, q, c.k, c.v, c.table, c.seqlens[:1])
    refused("weights", dec, q, c.k, c.v, c.table, c.seqlens, weights=c.w.half())
    refused("o must", dec, q, c.k, c.v, c.table, c.seqlens, out=q[:1])
    refused("lse", dec, q, c.k, c.v, c.table, c.seqlens, lse=torch.zeros(2, 4))
    refused("workspace", dec, q, c.k, c.v, c.table, c.seqlens, workspace=torch.zeros(1 << 20))
    k = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    refused("v must", fa.fa_paged_append, k, k[:, :2], c.k, c.v, c.table, c.seqlens)
    refused("w needs", fa.fa_paged_append, k, k, c.k, c.v, c.table, c.seqlens, w=c.w)
    refused("new_lens", fa.fa_paged_append, k, k, c.k, c.v, c.table, c.seqlens,
            new_lens=c.seqlens.long())
    refused("weights", fa.paged_evict, c.k, c.v, None, c.table, c.seqlens, c.table, 4, 1)
    refused("out_table", fa.paged_evict, c.k, c.v, c.w, c.table, c.seqlens, c.table[:1], 4, 1)
    refused("lse", fa.key_weights, k, k, torch.zeros(1, device="cuda"))
    refused("k must", fa.key_weights, k, k[:, :1], torch.zeros(1, device="cuda"))
    with pytest.raises(fa.FaError) as e:      # odd address
        x = torch.zeros(2 * 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 4, 64)
        dec(x, c.k, c.v, c.table, c.seqlens)
    assert e.value.code == -4
    with pytest.raises(fa.FaError) as e:      # workspace too small
        long = torch.cat([c.table, torch.full((2, 300), -1, dtype=torch.int32, device="cuda")], 1)
        dec(q, c.k, c.v, long, c.seqlens,
            workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -11
    with pytest.raises(fa.FaError) as e:      # o over q
        dec(q, c.k, c.v, c.table, c.seqlens, out=q)
    assert e.value.code == -5
    with pytest.raises(fa.FaError) as e:      # a budget that out_table cannot hold
        fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, c.table, 49, 1)
    assert e.value.code == -2
    lib, host = fa.load_library(), torch.zeros(2 * 4 * 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    rc = lib.fa_paged_decode(host.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), None,
                             c.table.data_ptr(), c.seqlens.data_ptr(), q.data_ptr(),
                             torch.zeros(8, device="cuda").data_ptr(), 2, 4, 2, 64, 16,
                             c.num_pages, c.max_pages, -1, 0.1, 0, ws.data_ptr(), ws.numel(), None)
    assert rc == -12                          # host memory


def test_serving_step_in_a_graph():
    """append + decode + the length's increment as one graph, replayed while the sequences grow
    over page borders, then an eviction graph, then more steps."""
    import io_aware_attention_fa2_gb300 as fa
    page, H, d = 16, 4, 128
    c = Cache([30, 3], page, H, d, "bf16", seed=5, weights=True, max_pages=6, spare=12)
    for b in range(2):                        # pages for the tokens to come
        used = -(-c.lens[b] // page)
        c.table[b, used:] = c.free[6 * b:6 * b + 6 - used].cuda()
    k1, v1 = (torch.zeros((2, 1, H, d), dtype=c.dtype, device="cuda") for _ in range(2))
    q1 = torch.zeros((2, 2 * H, d), dtype=c.dtype, device="cuda")
    o, lse = torch.zeros_like(q1), torch.zeros((2, 2 * H), device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")

    def step():
        c.seqlens.add_(one)
        fa.fa_paged_append(k1, v1, c.k, c.v, c.table, c.seqlens, weights=c.w)
        fa.paged_attention(q1, c.k, c.v, c.table, c.seqlens, weights=c.w, out=o, lse=lse)

    saved = [x.clone() for x in (c.k, c.v, c.w, c.seqlens)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for x, y in zip((c.k, c.v, c.w, c.seqlens), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((c.k, c.v, c.w, c.seqlens), saved):
        x.copy_(y)

    def run(times):
        for _ in range(times):
            k1.copy_(torch.randn(k1.shape, generator=c.g).to(c.dtype))
            v1.copy_(torch.randn(v1.shape, generator=c.g).to(c.dtype))
            q1.copy_(torch.randn(q1.shape, generator=c.g).to(c.dtype))
            before = c.w.clone()
            for b in range(2):                # the new token's weight starts at zero
                pg, row = c.table[b, c.lens[b] // page].long(), c.lens[b] % page
                before[pg, :, row] = 0
            graph.replay()
            c.lens = [n + 1 for n in c.lens]
            assert c.seqlens.tolist() == c.lens
            ref = decode_ref(c, q1, default_scale(d))
            check_decode(c, q1, o, lse, ref, c.lens)
            check_weights(c, before, ref)

    run(20)
    evict_graph = torch.cuda.CUDAGraph()
    out = c.table.clone()
    ref = evict_ref(c, out, 24, 6)
    with torch.cuda.graph(evict_graph):
        kept, lens = fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, out, 24, 6)
    evict_graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept.cpu(), ref[0])
    assert same_bits(c.k, ref[2]) and same_bits(c.v, ref[3]) and same_bits(c.w, ref[4])
    c.seqlens.copy_(lens)
    c.lens = lens.tolist()
    run(12)
