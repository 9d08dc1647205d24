"""Cases for speculative and branching decoding over the paged key-value cache: what each operator
reads, computes and returns, in elementary PyTorch operations, beside the framework's own calls
for the same thing.

Five operators:

  tree    attention of drafted tokens over the pages. The last n_b tokens of sequence b are
          drafted ones, a tree each: token i's parent is an earlier one or the context (-1). Token i
          sees the context, its ancestors and itself:
          O[b, i, h] = sum_j p_ij v_j,  p = softmax_j(scale <q_i, k_j>),  LSE = ln sum_j exp(...).
          A token stands at position context + depth; with a window only tokens at most `window`
          positions before it are seen. Without parents the drafted tokens are a chain.
  accept  after verification: the rows of the accepted tokens (an accepted one and its ancestors)
          moved behind the context in their order, and the new lengths.
  copy    rows of pages copied to other pages: keys, values and weights.
  fork    new sequences that continue others: whole pages are shared (counted in refs), the last
          one, where it is filled in part, gets a page from the pool and an entry in a list of copies.
  resize  the pages that sequences need for other lengths, taken from the pool or given back.

Cache layout: k_pages, v_pages [num_pages, page_size, Hkv, d]; weights [num_pages, Hkv, page_size]
fp32; block_table int32 [B, max_pages]: token t of sequence b is row t % page_size of page
block_table[b, t // page_size]; entries behind a sequence's last page hold -1. Pool: refs int32
[num_pages], how many tables a page stands in; free_pages int32 [num_pages], whose first
num_free[0] entries are the free pages, the last of them taken first.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # eight drafted tokens of one sequence with a short cache: latency
        dict(name="tree_b1_n1k_t8_d64", op="tree", B=1, Hq=8, Hkv=8, d=64, page=16, len=1001, T=8,
             dtype="fp16", chain=False, ragged=False, window=-1),
        # a serving batch of unequal lengths, small trees, four query heads to a key head
        dict(name="tree_b16_n16k_t16_gqa4", op="tree", B=16, Hq=32, Hkv=8, d=128, page=16,
             len=16384, T=16, dtype="bf16", chain=False, ragged=False, window=-1),
        # wide trees of 64 tokens over long caches
        dict(name="tree_b8_n32k_t64_gqa4", op="tree", B=8, Hq=32, Hkv=8, d=128, page=64,
             len=32768, T=64, dtype="bf16", chain=False, ragged=False, window=-1),
        # chains of up to five tokens (several heads that predict ahead), few key heads, very long
        dict(name="chain_b4_n64k_t5_gqa8", op="tree", B=4, Hq=32, Hkv=4, d=128, page=64,
             len=65536, T=5, dtype="fp16", chain=True, ragged=True, window=-1),
        # a sequence's accepted tokens: latency
        dict(name="accept_b1_t8", op="accept", B=1, Hkv=8, d=64, page=16, len=1001, T=8,
             dtype="fp16", weights=False),
        # a batch's, in a cache that keeps weights
        dict(name="accept_b64_t64", op="accept", B=64, Hkv=8, d=128, page=64, len=4096, T=64,
             dtype="bf16", weights=True),
        # the last pages of sixteen forked sequences: latency
        dict(name="copy_m16", op="copy", M=16, Hkv=8, d=128, page=16, dtype="bf16", weights=False,
             part=True),
        # a cache's worth of pages to other places
        dict(name="copy_m4k", op="copy", M=4096, Hkv=8, d=128, page=64, dtype="bf16", weights=True,
             part=False),
        # four samples from one prompt
        dict(name="fork_b1_c4", op="fork", B=1, C=4, page=16, len=1001),
        # beams of a batch of long sequences
        dict(name="fork_b64_c256", op="fork", B=64, C=256, page=16, len=32768),
        # room for the next drafted tokens of a batch, and back to what was accepted
        dict(name="resize_b16_t8", op="resize", B=16, page=16, len=4096, extra=8, grow=True),
        # a batch of long sequences that ends, and one that takes its place
        dict(name="resize_b256_n32k", op="resize", B=256, page=16, len=32768, extra=0, grow=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "copy", "fork", "resize"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    Hkv, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 5, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tree":
        n, T = _log(rng, 1, 65536), _log(rng, 1, 256)
        most = min(64, 8 * 32768 * 8 * 128 // (n * Hkv * d),              # bytes of the cache
                   8 * 64 * 32 * 32768 // (T * Hkv * G * (n + T)))        # pairs
        while most < 1:
            n, T = max(1, n // 2), max(1, T // 2)
            most = min(64, 8 * 32768 * 8 * 128 // (n * Hkv * d),
                       8 * 64 * 32 * 32768 // (T * Hkv * G * (n + T)))
        return dict(op=op, B=_log(rng, 1, most), Hq=Hkv * G, Hkv=Hkv, d=d, page=page, len=n, T=T,
                    dtype=dtype, chain=rng.random() < 0.3, ragged=rng.random() < 0.4,
                    window=rng.choice([-1, -1, -1, _log(rng, 1, n + 1)]))
    if op == "accept":
        n, T = _log(rng, 1, 8192), _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, max(1, min(64, 64 * 4096 * 8 // (n * Hkv)))), Hkv=Hkv,
                    d=d, page=page, len=n, T=T, dtype=dtype, weights=rng.random() < 0.5)
    if op == "copy":
        M = _log(rng, 1, max(1, min(4096, 4096 * 64 * 8 * 128 // (page * Hkv * d))))
        return dict(op=op, M=M, Hkv=Hkv, d=d, page=page, dtype=dtype, weights=rng.random() < 0.5,
                    part=rng.random() < 0.5)
    n, B = _log(rng, 1, 32768), _log(rng, 1, 256)
    if op == "fork":
        return dict(op=op, B=min(B, 64), C=_log(rng, 1, 256), page=page, len=n)
    return dict(op=op, B=B, page=page, len=n, extra=_log(rng, 1, 256), grow=rng.random() < 0.6)


def _lens(count, most, least=0):
    """One length for each sequence, up to `most`: the first is the longest, the others spread
    over the upper three quarters of the range. The same for every seed: work() goes by them."""
    r = random.Random("%s %s" % (count, most))
    return [most] + [max(least, r.randint(most // 4, most)) for _ in range(count - 1)]


def _drafts(case):
    return _lens(case["B"], case["T"], 1) if case.get("ragged") else [case["T"]] * case["B"]


def _pages(t, page):
    return -(-t // page)


def _table(page, g, lens, spare):
    """A block table over randomly ordered physical pages, the other pages, and their number."""
    width = max(_pages(n, page) for n in lens) or 1
    need = sum(_pages(n, page) for n in lens)
    order = torch.randperm(need + spare, generator=g, device=DEV).to(torch.int32)
    counts = torch.tensor([_pages(n, page) for n in lens], device=DEV)
    used = torch.arange(width, device=DEV)[None, :] < counts[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[used] = order[:need]
    return table, order[need:], need + spare


def _randn(g, shape, t, scale=1.0):
    """Normal values, made in slices so that the 32-bit ones never take much memory."""
    out = torch.empty(shape, dtype=t, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV) * scale
    return out


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _trees(g, B, T):
    """Parents of random trees: any earlier token, or the context."""
    i = torch.arange(T, device=DEV)
    u = torch.rand((B, T), generator=g, device=DEV)
    return torch.minimum((u * (i + 1)).long(), i).to(torch.int32) - 1


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st, page = dict(case), case["page"]
    if case["op"] in ("fork", "resize"):
        lens = _lens(case["B"], case["len"])
        if case["op"] == "fork":
            spare = case["C"] + 8
            st["source"] = torch.randint(0, case["B"], (case["C"],), generator=g,
                                         device=DEV).to(torch.int32)
            st["zero"] = torch.zeros_like(st["source"])
        else:
            later = [n + case["extra"] for n in lens] if case["grow"] else [0] * case["B"]
            spare = sum(max(0, _pages(m, page) - _pages(n, page))
                        for n, m in zip(lens, later)) + 8
            st["later"] = _int(later)
        st["table"], freed, count = _table(page, g, lens, spare)
        if case["op"] == "resize" and case["grow"]:
            # a serving table has columns for more tokens than its sequences hold
            st["table"] = torch.nn.functional.pad(
                st["table"], (0, _pages(case["extra"], page) + 1), value=-1).contiguous()
        st["seqlens"] = _int(lens)
        st["refs"] = torch.ones(count, dtype=torch.int32, device=DEV)
        st["refs"][freed.long()] = 0
        st["free"] = torch.full((count,), -1, dtype=torch.int32, device=DEV)
        st["free"][:freed.numel()] = freed
        st["num_free"] = _int([freed.numel()])
        return st
    t, d, Hkv = TYPES[case["dtype"]], case["d"], case["Hkv"]
    if case["op"] == "copy":
        M = case["M"]
        order = torch.randperm(2 * M, generator=g, device=DEV).to(torch.int32)
        st["src"], st["dst"], count = order[:M].contiguous(), order[M:].contiguous(), 2 * M
        st["rows"] = (torch.randint(1, page + 1, (M,), generator=g, device=DEV).to(torch.int32)
                      if case["part"] else None)
    else:
        B, T, new = case["B"], case["T"], _drafts(case)
        lens = [n + m for n, m in zip(_lens(B, case["len"]), new)]
        st["table"], _, count = _table(page, g, lens, 1)
        st["seqlens"] = _int(lens)
        st["new_lens"] = _int(new) if case.get("ragged") else None
        st["parents"] = None if case.get("chain") else _trees(g, B, T)
        if case["op"] == "accept":
            st["leaf"] = torch.randint(0, T, (B,), generator=g, device=DEV).to(torch.int32)
        else:
            st["scale"] = float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))
            st["q"] = _randn(g, (B, T, case["Hq"], d), t, 1.5)
    st["k_pages"], st["v_pages"] = (_randn(g, (count, page, Hkv, d), t) for _ in range(2))
    # accumulated attention weights: a heavy tail
    st["weights"] = (torch.exp(2.0 * torch.randn((count, Hkv, page), generator=g, device=DEV))
                     if case.get("weights") else None)
    return st


def run(st):
    return (_own if own else _plain)[st["op"]](st)


# --------------------------------------------------------------------------- the framework's calls
def _own_tree(st):
    import io_aware_attention_fa2_gb300 as fa
    return list(fa.paged_tree_attention(
        st["q"], st["k_pages"], st["v_pages"], st["table"], st["seqlens"], parents=st["parents"],
        new_lens=st["new_lens"], scale=st["scale"], window_left=st["window"]))


def _own_accept(st):
    import io_aware_attention_fa2_gb300 as fa
    path, lens = fa.paged_accept(st["k_pages"], st["v_pages"], st["table"], st["seqlens"],
                                 st["leaf"], st["parents"], weights=st["weights"])
    return [path, lens, st["k_pages"], st["v_pages"], st["weights"]]


def _own_copy(st):
    import io_aware_attention_fa2_gb300 as fa
    fa.fa_paged_copy(st["k_pages"], st["v_pages"], st["src"], st["dst"], rows=st["rows"],
                     weights=st["weights"])
    return [st["k_pages"], st["v_pages"], st["weights"]]


def _own_fork(st):
    import io_aware_attention_fa2_gb300 as fa
    pool = fa.PagePool(st["refs"], st["free"], st["num_free"])
    forked = fa.paged_fork(pool, st["table"], st["seqlens"], st["source"], st["page"])
    # the new sequences end again (in a table of their own, which their pages leave)
    ended = fa.paged_resize(pool, forked.block_table, forked.seqlens, st["zero"], st["page"])
    return [*forked, ended, st["refs"], st["free"], st["num_free"]]


def _own_resize(st):
    import io_aware_attention_fa2_gb300 as fa
    pool = fa.PagePool(st["refs"], st["free"], st["num_free"])
    there = fa.paged_resize(pool, st["table"], st["seqlens"], st["later"], st["page"])
    back = fa.paged_resize(pool, st["table"], there, st["seqlens"], st["page"])
    return [there, back, st["table"], st["refs"], st["free"], st["num_free"]]


_own = dict(tree=_own_tree, accept=_own_accept, copy=_own_copy, fork=_own_fork,
            resize=_own_resize)


# --------------------------------------------------------------------------- the plain forms
def _ancestors(parents):
    """[B, token, token]: whether the second is the first or an ancestor of it."""
    B, T = parents.shape
    see = (parents[:, :, None] == torch.arange(T, device=DEV)).float()
    see = see + torch.eye(T, device=DEV)
    n = 1
    while n < T:                                    # paths twice as long with every product
        see = (torch.matmul(see, see) > 0).float()
        n *= 2
    return see > 0


def _plain_tree(st):
    B, T, Hq, d = st["q"].shape
    Hkv, page, table = st["Hkv"], st["page"], st["table"].long().clamp(min=0)
    n = table.shape[1] * page
    t, i = torch.arange(n, device=DEV), torch.arange(T, device=DEV)
    new = st["new_lens"] if st["new_lens"] is not None else torch.full_like(st["seqlens"], T)
    base = (st["seqlens"] - new).long()
    anc = ((i[None, None, :] <= i[None, :, None]).expand(B, T, T) if st["parents"] is None
           else _ancestors(st["parents"]))
    depth = anc.sum(dim=2) - 1                                            # [B, T]
    # [B, token, key]: the context, and the drafted tokens that are ancestors
    node = (t[None, :] - base[:, None]).clamp(0, T - 1)
    draft = (t[None, :] >= base[:, None]) & (t[None, :] < st["seqlens"][:, None])
    see = (t[None, :] < base[:, None])[:, None, :] | (
        draft[:, None, :] & anc.gather(2, node[:, None, :].expand(B, T, n)))
    if st["window"] >= 0:
        place = torch.where(draft, base[:, None] + depth.gather(1, node), t[None, :])
        see = see & (place[:, None, :] >= (base[:, None] + depth)[:, :, None] - st["window"])
    see = (see & (i[None, :] < new[:, None])[:, :, None])[:, None, None]  # [B, 1, 1, T, n]
    q = st["q"].float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = st["k_pages"][table].view(B, n, Hkv, d).permute(0, 2, 3, 1).float()[:, :, None]
    s = torch.matmul(q, k).mul_(st["scale"])                              # [B, Hkv, G, T, key]
    s.masked_fill_(~see, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = p.sum(dim=-1, keepdim=True)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    v = st["v_pages"][table].view(B, n, Hkv, d).permute(0, 2, 1, 3).float()
    v = torch.where((t[None, :] < st["seqlens"][:, None])[:, None, :, None], v,
                    torch.zeros((), device=DEV))[:, :, None]
    o = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(st["q"].dtype)
    return [o, (m + torch.log(l)).reshape(B, Hq, T)]


def _slots(st, t):
    """Physical page and row of tokens t [B, n] of their sequences."""
    col = (t // st["page"]).clamp(0, st["table"].shape[1] - 1)
    return st["table"].gather(1, col).long().clamp(min=0), t % st["page"]


def _plain_accept(st):
    B, T = st["parents"].shape
    base = st["seqlens"].long() - T
    i = torch.arange(T, device=DEV)
    on = _ancestors(st["parents"]).gather(
        1, st["leaf"].long()[:, None, None].expand(B, 1, T))[:, 0]       # [B, T]
    count = on.sum(dim=1)
    path = torch.sort(torch.where(on, i[None, :], T), dim=1).values
    path = torch.where(path < T, path, -1)
    b, j = torch.nonzero(path >= 0, as_tuple=True)
    from_page, from_row = (x[b, j] for x in _slots(st, base[:, None] + path.clamp(min=0)))
    to_page, to_row = (x[b, j] for x in _slots(st, base[:, None] + i[None, :]))
    for pool in (st["k_pages"], st["v_pages"]):
        pool[to_page, to_row] = pool[from_page, from_row]
    if st["weights"] is not None:
        st["weights"][to_page, :, to_row] = st["weights"][from_page, :, from_row]
    return [path.to(torch.int32), (base + count).to(torch.int32), st["k_pages"], st["v_pages"],
            st["weights"]]


def _plain_copy(st):
    src, dst, page = st["src"].long(), st["dst"].long(), st["page"]
    if st["rows"] is None:
        for pool in (st["k_pages"], st["v_pages"], st["weights"]):
            if pool is not None:
                pool[dst] = pool[src]
    else:
        m, row = torch.nonzero(torch.arange(page, device=DEV)[None, :] < st["rows"][:, None],
                               as_tuple=True)
        for pool in (st["k_pages"], st["v_pages"]):
            pool[dst[m], row] = pool[src[m], row]
        if st["weights"] is not None:
            st["weights"][dst[m], :, row] = st["weights"][src[m], :, row]
    return [st["k_pages"], st["v_pages"], st["weights"]]


def _take(st, need):
    """need [n] pages for each of n askers: whether they fit, the place of each asker's first page
    in the order in which pages are taken, and the pool's number before."""
    total = torch.cumsum(need, dim=0)
    fits = (need == 0) | (total <= st["num_free"].long())
    had = st["num_free"].clone().long()
    st["num_free"] -= (need * fits).sum().to(torch.int32)
    return fits, total - need, had


def _plain_resize_of(st, table, old, later):
    """resize: releases first, in the tables' order, then takes."""
    page, width = st["page"], table.shape[1]
    a, z = (old.long() + page - 1) // page, (later.long() + page - 1) // page
    col = torch.arange(width, device=DEV)
    gone = (col[None, :] >= z[:, None]) & (col[None, :] < a[:, None])
    pages = table[gone].long()                                            # in order
    st["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    # a page is free with its last holder
    at = torch.arange(pages.numel(), device=DEV)
    last = torch.full(st["refs"].shape, -1, dtype=torch.long, device=DEV)
    last = last.scatter_reduce(0, pages, at, "amax")
    freed = pages[(last[pages] == at) & (st["refs"][pages] == 0)]
    have = st["num_free"].long()
    st["free"][have + torch.arange(freed.numel(), device=DEV)] = freed.to(torch.int32)
    st["num_free"] += freed.numel()
    table[gone] = -1
    need = (z - a).clamp(min=0)
    fits, first, had = _take(st, need)
    new = (col[None, :] >= a[:, None]) & (col[None, :] < z[:, None]) & fits[:, None]
    place = (first[:, None] + col[None, :] - a[:, None])[new]
    taken = st["free"][had - 1 - place]
    table[new] = taken
    st["refs"][taken.long()] = 1
    # what a taken page leaves on the stack does not matter: -1
    st["free"][torch.arange(st["free"].numel(), device=DEV) >= st["num_free"].long()] = -1
    return torch.where(fits, later, old)


def _plain_fork(st):
    page, source = st["page"], st["source"].long()
    n = st["seqlens"].long()[source]
    full, tail = n // page, n % page
    col = torch.arange(st["table"].shape[1], device=DEV)
    old = st["table"][source]
    fits, first, had = _take(st, (tail > 0).long())
    shared = (col[None, :] < full[:, None]) & fits[:, None]
    pages = old[shared].long()
    st["refs"].index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    copies = fits & (tail > 0)
    taken = st["free"][(had - 1 - first).clamp(min=0)]
    st["refs"][taken[copies].long()] = 1
    st["free"][torch.arange(st["free"].numel(), device=DEV) >= st["num_free"].long()] = -1
    table = torch.where(shared, old, -1)
    at = torch.nonzero(copies)[:, 0]
    table[at, full[at]] = taken[at]
    lens = torch.where(fits, n, -1).to(torch.int32)
    src = torch.where(copies, old.gather(1, full.clamp(max=col.numel() - 1)[:, None])[:, 0], -1)
    dst = torch.where(copies, taken, -1)
    rows = torch.where(copies, tail, 0).to(torch.int32)
    ended = _plain_resize_of(st, table, lens.clamp(min=0), st["zero"])
    return [table, lens, src, dst, rows, ended, st["refs"], st["free"], st["num_free"]]


def _plain_resize(st):
    there = _plain_resize_of(st, st["table"], st["seqlens"], st["later"])
    back = _plain_resize_of(st, st["table"], there, st["seqlens"])
    return [there, back, st["table"], st["refs"], st["free"], st["num_free"]]


_plain = dict(tree=_plain_tree, accept=_plain_accept, copy=_plain_copy, fork=_plain_fork,
              resize=_plain_resize)


# --------------------------------------------------------------------------- work and exact values
def work(case):
    page = case["page"]
    if case["op"] == "tree":
        d, Hq, Hkv, w = case["d"], case["Hq"], case["Hkv"], case["window"]
        pairs = seen = rows = 0
        for n, m in zip(_lens(case["B"], case["len"]), _drafts(case)):
            c = min(n, w) if w >= 0 else n      # of the context, by the tokens that follow it
            pairs += m * (c + 1)                # and at least itself
            seen += c + m
            rows += m
        return {"flops": 4.0 * pairs * Hq * d,
                "bytes": seen * Hkv * 4.0 * d + rows * Hq * (4.0 * d + 4)}
    if case["op"] == "accept":
        # the accepted tokens are a path: about ln T of a random tree
        rows = case["B"] * max(1.0, math.log(case["T"]))
        return {"flops": 0.0, "bytes": rows * case["Hkv"] * (8.0 * case["d"] + (
            8 if case["weights"] else 0)) + case["B"] * case["T"] * 8.0}
    if case["op"] == "copy":
        rows = case["M"] * (0.5 * (page + 1) if case["part"] else page)
        return {"flops": 0.0, "bytes": rows * case["Hkv"] * (8.0 * case["d"] + (
            8 if case["weights"] else 0))}
    lens = _lens(case["B"], case["len"])
    if case["op"] == "fork":
        # tables read and written, references raised and lowered again
        entries = case["C"] * sum(_pages(n, page) for n in lens) / case["B"]
        return {"flops": 0.0, "bytes": entries * 24.0 + case["C"] * 32.0}
    moved = sum(_pages(n + case["extra"], page) - _pages(n, page) if case["grow"]
                else _pages(n, page) for n in lens)
    # entries, references and the stack, there and back
    return {"flops": 0.0, "bytes": moved * 2 * 16.0 + case["B"] * 24.0}


def exact(case, seed):
    if case["op"] not in _exact:
        return None                     # whole numbers
    return _exact[case["op"]](case, prepare(case, seed))


def _line(parents, i):
    """Token i and its ancestors, from the tree's first: by walking up."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def _rows(st, b, n):
    """(page, row) of the first n tokens of sequence b."""
    page = st["page"]
    return (st["table"][b, :_pages(n, page)].long().repeat_interleave(page)[:n],
            torch.arange(n, device=DEV) % page)


def _exact_tree(case, st):
    B, T, Hq, Hkv, d = case["B"], case["T"], case["Hq"], case["Hkv"], case["d"]
    o = torch.zeros((B, T, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    trees = [list(range(-1, T - 1))] * B if st["parents"] is None else st["parents"].tolist()
    for b, (n, m) in enumerate(zip(st["seqlens"].tolist(), _drafts(case))):
        base = n - m
        bias = torch.full((m, n), -math.inf, dtype=torch.float64)
        for i in range(m):
            line = _line(trees[b], i)
            far = len(line) - 1 - case["window"] if case["window"] >= 0 else -n
            bias[i, max(0, base + far):base] = 0.0
            bias[i, [base + x for x in line[max(0, far):]]] = 0.0
        bias = bias.to(DEV)
        pg, row = _rows(st, b, n)
        for h in range(Hq):
            hk = h * Hkv // Hq
            s = st["q"][b, :m, h].double() @ st["k_pages"][pg, row, hk].double().T
            s = s * st["scale"] + bias
            lse[b, h, :m] = torch.logsumexp(s, dim=1)
            o[b, :m, h] = torch.softmax(s, dim=1) @ st["v_pages"][pg, row, hk].double()
    return [o, lse]


def _exact_accept(case, st):
    k, v = st["k_pages"].double(), st["v_pages"].double()
    w = None if st["weights"] is None else st["weights"].double()
    for b, n in enumerate(st["seqlens"].tolist()):
        base = n - case["T"]
        line = _line(st["parents"][b].tolist(), int(st["leaf"][b]))
        pg, row = _rows(st, b, n)
        src = torch.tensor([base + x for x in line], device=DEV)
        to = slice(base, base + len(line))
        k[pg[to], row[to]] = st["k_pages"][pg[src], row[src]].double()
        v[pg[to], row[to]] = st["v_pages"][pg[src], row[src]].double()
        if w is not None:
            w[pg[to], :, row[to]] = st["weights"][pg[src], :, row[src]].double()
    return [None, None, k, v, w]


def _exact_copy(case, st):
    out = []
    for name in ("k_pages", "v_pages", "weights"):
        x = None if st[name] is None else st[name].double()
        if x is not None:
            rows = case["page"] * torch.ones(case["M"], dtype=torch.int32, device=DEV) \
                if st["rows"] is None else st["rows"]
            keep = torch.arange(case["page"], device=DEV)[None, :] < rows[:, None]
            keep = keep[:, None, :] if name == "weights" else keep[:, :, None, None]
            for i in range(0, case["M"], 256):
                s, t = st["src"][i:i + 256].long(), st["dst"][i:i + 256].long()
                x[t] = torch.where(keep[i:i + 256], st[name][s].double(), st[name][t].double())
        out.append(x)
    return out


_exact = dict(tree=_exact_tree, accept=_exact_accept, copy=_exact_copy)
