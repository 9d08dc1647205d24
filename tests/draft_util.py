"""Drafted tokens and branching sequences in plain float64 and plain lists: the operators from
their definitions, and error bounds from the arithmetic the kernels are allowed."""
from __future__ import annotations

import math

import torch

from paged_util import Cache, score_error


def draft_cache(ctx, new, page, Hkv, d, dtype, **kw):
    """A Cache whose sequences have ctx[b] tokens of context and new[b] drafted ones."""
    return Cache([n + m for n, m in zip(ctx, new)], page, Hkv, d, dtype, **kw)


def random_trees(g, B, T, kind="random"):
    """int32 [B, T] parents."""
    out = torch.full((B, T), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(T):
            if kind == "chain":
                out[b, i] = i - 1
            elif kind == "random":
                out[b, i] = int(torch.randint(-1, max(i, 0), (1,), generator=g)) if i else -1
            elif kind == "deep":
                out[b, i] = max(-1, i - 1 - int(torch.randint(0, 2, (1,), generator=g)))
    return out


def line(parents, i):
    """Token i and its ancestors, ascending; a parent that is no earlier token counts as -1."""
    path = []
    while i >= 0:
        path.append(i)
        up = i - 1 if parents is None else int(parents[i])
        i = up if -1 <= up < i else -1
    return path[::-1]


def seen_tokens(base, parents, i, window):
    """Tokens of the sequence that drafted token i sees."""
    path = line(parents, i)
    pos = base + len(path) - 1
    lo = pos - window if window >= 0 else 0
    return list(range(max(0, lo), base)) + [base + a for x, a in enumerate(path) if base + x >= lo]


def tree_ref(c: Cache, q, scale, parents=None, new=None, window=-1, drop=None, lens=None):
    """float64 (O, LSE, bounds of each) of q [B, T, Hq, d]. `drop`: predicate of (b, token) whose
    tokens are left out."""
    B, T, Hq, d = q.shape
    G = Hq // c.Hkv
    half = torch.finfo(c.dtype).eps / 2
    table, K, V = c.table.cpu(), c.k.cpu().double(), c.v.cpu().double()
    q = q.cpu().double()
    o = torch.zeros((B, T, Hq, d), dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    for b, n in enumerate(lens or c.lens):
        m = T if new is None else min(max(new[b], 0), T)
        base = n - m
        if base < 0 or n > c.max_pages * c.page or m == 0:
            continue
        tree = None if parents is None else parents[b].tolist()
        see = torch.zeros((m, max(n, 1)), dtype=torch.bool)
        for i in range(m):
            see[i, seen_tokens(base, tree, i, window)] = True
        if drop is not None:
            for t in range(n):
                if drop(b, t):
                    see[:, t] = False
        t = torch.arange(n)
        pg, row = table[b, t // c.page].long().clamp(0, c.num_pages - 1), t % c.page
        hide = torch.zeros((), dtype=torch.float64)
        for h in range(Hq):
            k, v = K[pg, row, h // G], V[pg, row, h // G]
            s = torch.where(see, q[b, :m, h] @ k.nan_to_num().T * scale, -math.inf)
            e = score_error(q[b, :m, h][:, None], k.nan_to_num()[None], scale)
            e = torch.where(see, e, hide).amax(1)
            any_seen = see.any(1)
            z = torch.where(any_seen, torch.logsumexp(s, 1), hide)
            p = torch.where(see, torch.exp(s - z[:, None]), hide)
            v = v.nan_to_num()
            pv, sv = p @ v.abs(), see.double() @ v.abs()
            out = p @ v
            o[b, :m, h] = out
            # every p off by exp(+-2e) at most (its score and the sum's), 2^-19 for exp2, the sums
            # and the joins; P is rounded to the type once (fp16, which ends at 2^-24, holds it
            # 2^11 times as large at least: 2^-36 a token); the output is rounded once
            small = 2.0 ** -36 if c.dtype == torch.float16 else 0.0
            ob[b, :m, h] = (half * out.abs() + (half + 2.0 * e[:, None] + 2.0 ** -19) * pv * 1.01
                            + small * sv + 1e-7)
            lse[b, h, :m] = torch.where(any_seen, z, -math.inf)
            lb[b, h, :m] = e + 2.0 ** -20 + 2.0 ** -22 * z.abs()
    return o, lse, ob, lb


def check_tree(o, lse, ref, what, finite=True):
    o_ref, lse_ref, ob, lb = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    if finite:
        assert torch.isfinite(o).all(), what
    bad = (o - o_ref).abs() - ob
    assert (bad <= 0).all(), (what, float(bad.max()))
    empty = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), empty), what
    assert ((lse - lse_ref).abs()[~empty] <= lb[~empty]).all(), what


def accept_ref(c: Cache, parents, leaf, T, new=None):
    """path, new lengths and the pools after an accept of well-formed arguments."""
    B, table = len(c.lens), c.table.cpu()
    k, v = c.k.cpu().clone(), c.v.cpu().clone()
    w = None if c.w is None else c.w.cpu().clone()
    old = [None if x is None else x.clone() for x in (k, v, w)]
    path = torch.full((B, T), -1, dtype=torch.int32)
    lens = []
    for b, n in enumerate(c.lens):
        m = T if new is None else min(max(new[b], 0), T)
        base = n - m
        keep = line(None if parents is None else parents[b].tolist(), int(leaf[b]))
        path[b, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
        lens.append(base + len(keep))
        for j, i in enumerate(keep):
            sp, sr = int(table[b, (base + i) // c.page]), (base + i) % c.page
            dp, dr = int(table[b, (base + j) // c.page]), (base + j) % c.page
            k[dp, dr], v[dp, dr] = old[0][sp, sr], old[1][sp, sr]
            if w is not None:
                w[dp, :, dr] = old[2][sp, :, sr]
    return path, torch.tensor(lens, dtype=torch.int32), k, v, w


class Pool:
    """The books of a pool in plain lists, and the operators on them."""

    def __init__(self, num_pages):
        self.refs = [0] * num_pages
        self.free = list(range(num_pages))[::-1]

    def take(self):
        page = self.free.pop()
        self.refs[page] = 1
        return page

    def stack(self):
        return self.free + [-1] * (len(self.refs) - len(self.free))

    def resize(self, table, old, later, page):
        """In place on table (lists); returns granted."""
        given, holders = [], {}
        for b, row in enumerate(table):
            a, z = -(-old[b] // page), -(-later[b] // page)
            for col in range(z, a):
                given.append(row[col])
                holders[row[col]] = len(given) - 1
                self.refs[row[col]] -= 1
                row[col] = -1
        for f, pg in enumerate(given):
            if holders[pg] == f and self.refs[pg] == 0:
                self.free.append(pg)
        granted, room = [], len(self.free)
        for b, row in enumerate(table):
            a, z = -(-old[b] // page), -(-later[b] // page)
            need = max(0, z - a)
            room -= need
            if need and room < 0:
                granted.append(old[b])
                continue
            for col in range(a, z):
                row[col] = self.take()
            granted.append(later[b])
        return granted

    def fork(self, table, lens, source, page):
        """(tables, lengths, copies' src, dst, rows) of the new sequences."""
        out = ([], [], [], [], [])
        for s in source:
            n = 0 if s < 0 else lens[s]
            row, copy = [-1] * len(table[0]), (-1, -1, 0)
            if n % page and not self.free:
                n = -1
            elif n:
                for col in range(n // page):
                    row[col] = table[s][col]
                    self.refs[row[col]] += 1
                if n % page:
                    row[n // page] = self.take()
                    copy = (table[s][n // page], row[n // page], n % page)
            for x, y in zip(out, (row, n, *copy)):
                x.append(y)
        return out
