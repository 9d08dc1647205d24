"""The paged cache in plain float64: caches with poisoned spare rows, the operators from their
definitions, and error bounds from the arithmetic the kernels are allowed."""
from __future__ import annotations

import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Cache:
    """A pool whose rows outside every sequence hold `poison` (NaN unless given)."""

    def __init__(self, lens, page, Hkv, d, dtype, seed=0, weights=False, max_pages=None, spare=3,
                 poison=float("nan"), device="cuda", capacity_tail=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.page, self.Hkv, self.d, self.dtype = g, page, Hkv, d, DT[dtype]
        used = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(1, max(used) + capacity_tail)
        self.num_pages = sum(used) + spare
        order = torch.randperm(self.num_pages, generator=g)
        table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u].to(torch.int32)
            at += u
        self.free = order[at:].to(torch.int32)
        self.lens = list(lens)
        shape = (self.num_pages, page, Hkv, d)
        k = torch.full(shape, poison, dtype=self.dtype)
        v = torch.full(shape, poison, dtype=self.dtype)
        w = torch.full((self.num_pages, Hkv, page), poison, dtype=torch.float32)
        for b, n in enumerate(lens):
            pg, row = self.rows(table, b, n)
            k[pg, row] = torch.randn((n, Hkv, d), generator=g).to(self.dtype)
            v[pg, row] = torch.randn((n, Hkv, d), generator=g).to(self.dtype)
            w[pg, :, row] = torch.rand((n, Hkv), generator=g)
        self.table, self.k, self.v = table.to(device), k.to(device), v.to(device)
        self.w = w.to(device) if weights else None
        self.seqlens = torch.tensor(lens, dtype=torch.int32, device=device)

    def rows(self, table, b, n):
        pg = table[b, :max(1, -(-n // self.page))].long().repeat_interleave(self.page)[:n]
        return pg, torch.arange(n, device=table.device) % self.page

    def query(self, Hq, scale=1.0):
        q = torch.randn((len(self.lens), Hq, self.d), generator=self.g) * scale
        return q.to(self.dtype).to(self.k.device)


def default_scale(d):
    return float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))


def score_error(q, k, scale):
    """Most that a score scale * <q, k> can be off when its products are exact and its sum of d
    terms runs in 32 bits with a step of 2^-23 each (which allows for truncation), plus the
    rounding of scale * log2(e) and of the product with it: relative 2^-23 of the sum of
    absolute values once more. q [.., d] and k [.., d] broadcast."""
    d = q.shape[-1]
    return abs(scale) * (d + 2) * 2.0 ** -23 * (q.abs() * k.abs()).sum(-1)


def decode_ref(c: Cache, q, scale, window=-1, lens=None, drop=None):
    """float64 (O, LSE, added weights [B][Hkv, n] list, bounds of each). `drop`: predicate of
    (b, token) whose tokens are left out."""
    B, Hq, d = q.shape
    G = Hq // c.Hkv
    half = torch.finfo(c.dtype).eps / 2
    table, K, V = c.table.cpu(), c.k.cpu().double(), c.v.cpu().double()
    q = q.cpu().double()
    o = torch.zeros((B, Hq, d), dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    added, added_b = [], []
    for b, n in enumerate(lens or c.lens):
        lo = max(0, n - 1 - window) if window >= 0 else 0
        t = [x for x in range(lo, n) if drop is None or not drop(b, x)]
        add = torch.zeros((c.Hkv, n), dtype=torch.float64)
        addb = torch.zeros_like(add)
        if t:
            t = torch.tensor(t)
            pg, row = table[b, t // c.page].long(), t % c.page
            for h in range(Hq):
                k, v = K[pg, row, h // G], V[pg, row, h // G]
                s = k @ q[b, h] * scale
                e = float(score_error(q[b, h], k, scale).max())
                lse[b, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[b, h])
                o[b, h] = p @ v
                # every p off by exp(+-2e) at most (its score and the sum's), 2^-20 for exp2 and
                # the sums; P may be rounded to the type once; the output is rounded once
                pv = p @ v.abs()
                ob[b, h] = half * o[b, h].abs() + (half + 2.0 * e + 2.0 ** -19) * pv * 1.01 + 1e-7
                lb[b, h] = e + 2.0 ** -20 + 2.0 ** -22 * lse[b, h].abs()
                add[h // G, t] += p
                addb[h // G, t] += p * (2.0 * e + 2.0 ** -18 + 2.0 ** -22 * lse[b, h].abs())
        added.append(add)
        added_b.append(addb)
    return o, lse, added, ob, lb, added_b


def check_decode(c, q, o, lse, ref, what):
    o_ref, lse_ref, _, ob, lb, _ = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), what
    assert ((o - o_ref).abs() <= ob).all(), (what, float(((o - o_ref).abs() - ob).max()))
    empty = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), empty), what
    assert ((lse - lse_ref).abs()[~empty] <= lb[~empty]).all(), what


def key_weights_ref(q, k, lse, scale, causal=False, window=(-1, -1), lens=None):
    """float64 w [B, Hkv, N] and a bound on a kernel's error."""
    q, k, lse = q.cpu().double(), k.cpu().double(), lse.cpu().double()
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    i = torch.arange(N)
    w = torch.zeros((B, Hkv, N), dtype=torch.float64)
    wb = torch.zeros_like(w)
    for b in range(B):
        n = N if lens is None else min(max(lens[b], 0), N)
        see = (i[None] < n) & (i[:, None] < n)
        if causal:
            see &= i[None] <= i[:, None]
        if window[0] >= 0:
            see &= i[None] >= i[:, None] - window[0]
        if window[1] >= 0:
            see &= i[None] <= i[:, None] + window[1]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            qq, kk = q[b, :, h].nan_to_num(), k[b, :, hk].nan_to_num()
            s = qq @ kk.T * scale
            e = abs(scale) * (d + 2) * 2.0 ** -23 * (qq.abs() @ kk.abs().T)
            p = torch.where(see, torch.exp(s - lse[b, h, :, None]), torch.zeros((), dtype=s.dtype))
            p = torch.where(torch.isneginf(lse[b, h])[:, None], torch.zeros_like(p), p)
            w[b, hk] += p.sum(0)
            # the score's error, LSE * log2(e) and the difference rounded in 32 bits, exp2, and
            # sums of up to N * G terms in chunks of at most 2048 (2^-24 a step)
            r = e + 2.0 ** -22 * (lse[b, h, :, None].abs().nan_to_num(posinf=0) + s.abs()) + 2.0 ** -13
            wb[b, hk] += (p * r).sum(0)
    return w, wb + 1e-30


def evict_ref(c: Cache, out_table, budget, recent):
    """kept [B, Hkv, budget], new lengths and the pools after eviction, by sorting; bad or
    refused sequences are not covered here."""
    table, out = c.table.cpu(), out_table.cpu()
    k, v, w = c.k.cpu().clone(), c.v.cpu().clone(), c.w.cpu().clone()
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    kept = torch.full((len(c.lens), c.Hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        m = min(n, budget)
        if m == 0:
            continue
        pg, row = c.rows(table, b, n)
        to = out[b].long().repeat_interleave(c.page)[:m]
        to_row = torch.arange(m) % c.page
        old = n - recent if n > budget else 0
        for h in range(c.Hkv):
            if n <= budget:
                keep = list(range(n))
            else:
                value = w0[pg, h, row].double().tolist()[:old]
                rank = sorted(range(old), key=lambda t: (
                    math.inf if math.isnan(value[t]) else -value[t],
                    math.isnan(value[t]), t))
                keep = sorted(rank[:budget - recent]) + list(range(old, n))
            keep = torch.tensor(keep)
            kept[b, h, :m] = keep.to(torch.int32)
            k[to, to_row, h], v[to, to_row, h] = k0[pg[keep], row[keep], h], v0[pg[keep], row[keep], h]
            w[to, h, to_row] = w0[pg[keep], h, row[keep]]
    return kept, torch.tensor([min(n, budget) for n in c.lens], dtype=torch.int32), k, v, w


def same_bits(a, b):
    """Equal bit for bit, NaN included."""
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.cpu().view(kind), b.cpu().view(kind))
