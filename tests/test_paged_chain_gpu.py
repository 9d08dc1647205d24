"""The paged cache's kernels may be launched before the work in front of them ends. Whole chains of
calls, behind work that has just written what they read, against the same calls made one by one
with the device idle in between, and those against float64."""
import pytest
import torch

from paged_util import (Cache, check_decode, decode_ref, default_scale, evict_ref, key_weights_ref,
                        same_bits)
from test_paged_gpu import check_weights, free_table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


class Chain:
    """Key weights, an append, a decode with weights, an eviction and a decode of what it kept, on
    one set of buffers; `inputs[i]` are different contents for them."""

    def __init__(self, d, dtype, Hq, Hkv, page):
        self.scale, self.budget, self.recent = default_scale(d), 256, 31
        self.inputs = []
        for seed in range(3):
            c = Cache([3000 + 400 * seed, 900 - seed], page, Hkv, d, dtype, seed=seed, weights=True,
                      spare=2 * 256 // page, max_pages=4000 // page + 1)
            self.num_pages = 5600 // page
            k, v, w = (torch.zeros((self.num_pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
                       for x in (c.k, c.v, c.w))
            k[:c.num_pages], v[:c.num_pages], w[:c.num_pages] = c.k, c.v, c.w
            q = torch.randn((2, 260, Hq, d), generator=c.g).to(c.dtype).cuda()
            p = torch.randn((2, 260, Hkv, d), generator=c.g).to(c.dtype).cuda()
            lse = (6.0 + torch.rand((2, Hq, 260), generator=c.g)).cuda()
            new = torch.tensor([200 + seed, 17], dtype=torch.int32, device="cuda")
            self.inputs.append(dict(c=c, t=[q[:, 0].clone(), k, v, w, c.table, c.seqlens,
                                            free_table(c, self.budget), q, p, lse, new]))
        self.t = [torch.zeros_like(x) for x in self.inputs[0]["t"]]
        self.kw = torch.zeros((2, Hkv, 260), device="cuda")
        self.o, self.o2 = torch.zeros_like(self.t[0]), torch.zeros_like(self.t[0])
        self.lse, self.lse2 = (torch.zeros((2, Hq), device="cuda") for _ in range(2))
        self.kept = torch.zeros((2, Hkv, self.budget), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(2, dtype=torch.int32, device="cuda")

    def fill(self, i, kernel):
        """Contents i into the buffers, by copies or by kernels (on the bits)."""
        for x, y in zip(self.t, self.inputs[i]["t"]):
            if kernel:
                kind = torch.int16 if x.element_size() == 2 else torch.int32
                torch.bitwise_or(y.view(kind), 0, out=x.view(kind))
            else:
                x.copy_(y)

    def calls(self, between=lambda: None):
        import io_aware_attention_fa2_gb300 as fa
        q1, k, v, w, table, lens, out, q, p, lse, new = self.t
        fa.fa_key_weights(q, p, lse, self.kw, True, self.scale)
        between()
        fa.fa_paged_append(p, p, k, v, table, lens, new_lens=new, w=self.kw, weights=w)
        between()
        fa.fa_paged_decode(q1, k, v, table, lens, self.o, self.lse, self.scale, weights=w)
        between()
        fa.fa_paged_evict(k, v, w, table, lens, out, self.kept, self.lens, self.recent)
        between()
        fa.fa_paged_decode(q1, k, v, out, self.lens, self.o2, self.lse2, self.scale)
        between()

    def results(self):
        return [x.clone() for x in (self.kw, *self.t[1:4], self.o, self.lse, self.kept, self.lens,
                                    self.o2, self.lse2)]


def check_one_by_one(chain, i):
    """The calls on contents i, each on an idle device, against float64; their results."""
    import io_aware_attention_fa2_gb300 as fa
    c, scale = chain.inputs[i]["c"], chain.scale
    chain.fill(i, False)
    torch.cuda.synchronize()
    q1, k, v, w, table, lens, out, q, p, lse, new = chain.t
    c.num_pages = chain.num_pages
    n = new.tolist()
    snaps = []

    def between():
        torch.cuda.synchronize()
        snaps.append([x.clone() for x in (k, v, w)])

    chain.calls(between)
    ref, bound = key_weights_ref(q, p, lse, scale, True)
    assert ((chain.kw.double().cpu() - ref).abs() <= bound).all()
    c.k, c.v, c.w = (x.clone() for x in chain.inputs[i]["t"][1:4])
    for b in range(2):
        pg, row = (x[c.lens[b] - n[b]:] for x in c.rows(c.table, b, c.lens[b]))
        c.k[pg, row] = c.v[pg, row] = p[b, :n[b]]
        c.w[pg, :, row] = chain.kw[b, :, :n[b]].T
    for got, want in zip(snaps[1], (c.k, c.v, c.w)):
        assert same_bits(got, want)
    ref = decode_ref(c, q1, scale)
    check_decode(c, q1, chain.o, chain.lse, ref, "first decode")
    before, c.w = c.w, snaps[2][2]
    check_weights(c, before, ref)
    kept, new_lens, *pools = evict_ref(c, out, chain.budget, chain.recent)
    assert torch.equal(chain.kept.cpu(), kept) and torch.equal(chain.lens.cpu(), new_lens)
    for got, want in zip(snaps[3], pools):
        assert same_bits(got, want)
    c.k, c.v, c.table, lens_before, c.lens = *snaps[3][:2], out, c.lens, new_lens.tolist()
    check_decode(c, q1, chain.o2, chain.lse2, decode_ref(c, q1, scale), "second decode")
    assert fa.device_error() == 0
    return chain.results()


@pytest.mark.parametrize("d,dtype,Hq,Hkv,page", [(64, "bf16", 8, 2, 16), (128, "fp16", 3, 3, 64)])
def test_chains_give_what_single_calls_give(d, dtype, Hq, Hkv, page):
    chain = Chain(d, dtype, Hq, Hkv, page)
    want = [check_one_by_one(chain, i) for i in range(3)]
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def run(i, kernel):
        big.zero_()                       # work that is still running when the chain is enqueued
        chain.fill(i, kernel)
        chain.calls()

    for how in ("stream", "streams", "graph"):
        for kernel in (False, True):
            if how == "graph":
                graphs = []
                for i in range(3):
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g):
                        run(i, kernel)
                    graphs.append(g)
            # other contents each time, with nothing waited for in between: what a kernel read too
            # early would be those of the run before
            got = []
            for i in (0, 1, 2, 1, 0, 2):
                if how == "graph":
                    graphs[i].replay()
                elif how == "streams":
                    side = torch.cuda.Stream()
                    side.wait_stream(torch.cuda.current_stream())
                    with torch.cuda.stream(side):
                        big.zero_()
                        chain.fill(i, kernel)
                    torch.cuda.current_stream().wait_stream(side)
                    chain.calls()
                else:
                    run(i, kernel)
                got.append((i, chain.results()))
            torch.cuda.synchronize()
            for i, results in got:
                for x, y in zip(results, want[i]):
                    assert same_bits(x, y), (how, kernel, i)
