"""Cases for the paged key-value cache and its neighbours: what each operator reads, computes and
returns, in elementary PyTorch operations, beside the framework's own calls for the same thing.

Four operators, the life of a key-value cache that is kept within a budget:

  key_weights  the attention weight that every key of a prompt received, summed over its queries
               and over the query heads that share the key's head:
               w[b, hk, j] = sum_{h in group hk} sum_i exp(scale <q_i, k_j> - LSE[b, h, i]),
               over the queries i that see key j.
  append       new keys and values (and their weights) written into the pages of a cache.
  decode       attention of one new token over the pages:
               O[b, h] = sum_j p_j v_j,  p = softmax_j(scale <q, k_j>),  LSE = ln sum_j exp(...);
               when the cache keeps weights, weights[j] += sum_{h in group} p_j.
  evict        the `recent` newest tokens and the heaviest others, `budget` in all for every head,
               moved to the front pages in their order.

Cache layout: k_pages, v_pages [num_pages, page_size, Hkv, d]; weights [num_pages, Hkv, page_size]
fp32; block_table int32 [B, max_pages]: token t of sequence b is row t % page_size of page
block_table[b, t // page_size]; entries behind a sequence's last page hold -1.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a short prompt's weights, odd length: latency
        dict(name="weights_n500_d64", op="key_weights", B=1, Hq=8, Hkv=8, N=500, d=64,
             dtype="fp16", causal=True, window=-1, padded=False),
        # a batch of ordinary prompts, padded to the longest
        dict(name="weights_b4_n1k_d128", op="key_weights", B=4, Hq=16, Hkv=16, N=1024, d=128,
             dtype="bf16", causal=True, window=-1, padded=True),
        # a long prompt whose query heads share key heads
        dict(name="weights_n8k_d128_gqa", op="key_weights", B=2, Hq=16, Hkv=4, N=8192, d=128,
             dtype="bf16", causal=True, window=-1, padded=False),
        # the longest prompt
        dict(name="weights_n16k_d128", op="key_weights", B=1, Hq=16, Hkv=16, N=16384, d=128,
             dtype="bf16", causal=True, window=-1, padded=False),
        # one token of each sequence of a batch: latency
        dict(name="append_token_b16", op="append", B=16, Hkv=8, N=1, d=128, page=16,
             dtype="bf16", weights=False, start=5000),
        # ragged prompts into the pages, with their weights
        dict(name="append_prompt_b4_n8k", op="append", B=4, Hkv=16, N=8192, d=128, page=64,
             dtype="bf16", weights=True, start=0),
        # one sequence, short cache: latency
        dict(name="decode_b1_n1k_d64", op="decode", B=1, Hq=8, Hkv=8, d=64, page=16, len=1001,
             dtype="fp16", weights=False, window=-1),
        # a serving batch of unequal lengths, four query heads to a key head
        dict(name="decode_b16_n16k_gqa4", op="decode", B=16, Hq=32, Hkv=8, d=128, page=16,
             len=16384, dtype="bf16", weights=False, window=-1),
        # few heads, a very long cache: only a split over its length fills the GPU
        dict(name="decode_b4_n64k_gqa8", op="decode", B=4, Hq=32, Hkv=4, d=128, page=64,
             len=65536, dtype="bf16", weights=False, window=-1),
        # the same step in a cache that keeps the weights its tokens received
        dict(name="decode_w_b8_n32k_gqa4", op="decode", B=8, Hq=32, Hkv=8, d=128, page=32,
             len=32768, dtype="bf16", weights=True, window=-1),
        # one sequence over its budget: latency
        dict(name="evict_b1_n1200", op="evict", B=1, Hkv=8, d=64, page=16, len=1200,
             budget=1024, recent=128, dtype="fp16"),
        # long sequences down to an eighth
        dict(name="evict_b8_n32k", op="evict", B=8, Hkv=8, d=128, page=64, len=32768,
             budget=4096, recent=512, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["key_weights", "append", "decode", "evict"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    Hkv, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "key_weights":
        Hq, causal = Hkv * min(G, 32 // Hkv), rng.random() < 0.8
        pairs = 16 * 16384 ** 2 * (1.0 if causal else 0.5) / Hq    # of query and key, most
        N = _log(rng, 1, min(16384, int(pairs ** 0.5)))
        B = _log(rng, 1, min(16, int(pairs / (N * N))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, dtype=dtype, causal=causal,
                    window=rng.choice([-1, -1, -1, _log(rng, 1, 4096)]),
                    padded=rng.random() < 0.3)
    if op == "append":
        N = rng.choice([1, _log(rng, 1, 8192)])
        B = _log(rng, 1, min(64, 4 * 8192 * 16 * 128 // (N * Hkv * d)))
        return dict(op=op, B=B, Hkv=Hkv, N=N, d=d, page=page, dtype=dtype,
                    weights=rng.random() < 0.5, start=rng.choice([0, _log(rng, 1, 4096)]))
    if op == "decode":
        n = _log(rng, 1, 65536)
        B = _log(rng, 1, min(64, 8 * 32768 * 8 * 128 // (n * Hkv * d)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, len=n, dtype=dtype,
                    weights=rng.random() < 0.4, window=rng.choice([-1, -1, -1, _log(rng, 1, n)]))
    n = _log(rng, 2, 65536)
    budget = min(4096, _log(rng, 1, n))
    B = _log(rng, 1, max(1, min(16, 8 * 32768 * 8 // (n * Hkv), 8 * 4096 * 8 // (budget * Hkv))))
    return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, len=n, budget=budget,
                recent=rng.randint(0, budget), dtype=dtype)


def _lens(case, most, least=0):
    """One length for each sequence, up to `most`: the first is the longest, the others spread
    over the upper three quarters of the range. The same for every seed: work() goes by them."""
    r = random.Random("%s %s" % (case["B"], most))
    return [most] + [max(least, r.randint(most // 4, most)) for _ in range(case["B"] - 1)]


def _key_lens(case):
    return _lens(case, case["N"], 1) if case["padded"] else [case["N"]] * case["B"]


def _pages(t, page):
    return -(-t // page)


def _table(case, g, lens, spare=0):
    """A block table over randomly ordered physical pages, and the number of pages of the pool."""
    page = case["page"]
    width = max(_pages(n, page) for n in lens) or 1
    need = sum(_pages(n, page) for n in lens)
    order = torch.randperm(need + spare + 1, generator=g, device=DEV).to(torch.int32)
    counts = torch.tensor([_pages(n, page) for n in lens], device=DEV)
    col = torch.arange(width, device=DEV)
    used = col[None, :] < counts[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[used] = order[:need]
    return table, need + spare + 1, order[need:need + spare]


def _randn(g, shape, t, scale=1.0):
    """Normal values, made in slices so that the 32-bit ones never take much memory."""
    out = torch.empty(shape, dtype=t, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV) * scale
    return out


def _received(g, shape):
    """Accumulated attention weights: a heavy tail, and exact zeros for tokens never looked at."""
    w = torch.exp(2.0 * torch.randn(shape, generator=g, device=DEV) - 2.0)
    return torch.where(w < 0.01, torch.zeros_like(w), w)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t, d, Hkv, B = TYPES[case["dtype"]], case["d"], case["Hkv"], case["B"]
    st = dict(case)
    st["scale"] = float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))
    if case["op"] == "key_weights":
        N, Hq = case["N"], case["Hq"]
        st["q"] = _randn(g, (B, N, Hq, d), t, 1.5)
        st["k"] = _randn(g, (B, N, Hkv, d), t)
        lens = _key_lens(case)
        st["seqlens"] = torch.tensor(lens, dtype=torch.int32, device=DEV) if case["padded"] else None
        # the log-sum-exp that the prompt's forward left behind
        i = torch.arange(N, device=DEV)
        lse = torch.empty((B, Hq, N), device=DEV)
        for b in range(B):
            see = _visible(i, case, lens[b])
            for h in range(Hq):
                s = st["q"][b, :, h].float() @ st["k"][b, :, h // (Hq // Hkv)].float().T
                s = (s * st["scale"]).masked_fill_(~see, -math.inf)
                lse[b, h] = torch.logsumexp(s, dim=-1)
        st["lse"] = lse
        return st
    if case["op"] == "append":
        ends = [case["start"] + n for n in _lens(case, case["N"], 1)]
        table, pool, _ = _table(case, g, ends)
        st["seqlens"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        st["new_lens"] = st["seqlens"] - case["start"]
        st["k"], st["v"] = (_randn(g, (B, case["N"], Hkv, d), t) for _ in range(2))
        st["w"] = _received(g, (B, Hkv, case["N"])) if case["weights"] else None
    else:
        lens = _lens(case, case["len"])
        # the freed pages that an eviction moves the kept tokens into
        spare = B * _pages(case["budget"], case["page"]) if case["op"] == "evict" else 0
        table, pool, freed = _table(case, g, lens, spare)
        st["seqlens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["table"] = table
    st["k_pages"], st["v_pages"] = (_randn(g, (pool, case["page"], Hkv, d), t) for _ in range(2))
    keeps = case["op"] == "evict" or case["weights"]
    st["weights"] = _received(g, (pool, Hkv, case["page"])) if keeps else None
    if case["op"] == "decode":
        st["q"] = _randn(g, (B, case["Hq"], d), t, 1.5)
    if case["op"] == "evict":
        st["out_table"] = freed.view(B, -1)
    return st


def _visible(i, case, n):
    """[query, key]: which keys a prompt's query sees; queries behind the sequence's end count
    for nothing."""
    see = (i[None, :] < n) & (i[:, None] < n)
    if case["causal"]:
        see &= i[None, :] <= i[:, None]
    if case["window"] >= 0:
        see &= i[None, :] >= i[:, None] - case["window"]
    return see


def run(st):
    return (_own if own else _plain)[st["op"]](st)


# --------------------------------------------------------------------------- the framework's calls
def _own_key_weights(st):
    import io_aware_attention_fa2_gb300 as fa
    return fa.key_weights(st["q"], st["k"], st["lse"], causal=st["causal"], scale=st["scale"],
                          window=(st["window"], -1), seqlens_k=st["seqlens"])


def _own_append(st):
    import io_aware_attention_fa2_gb300 as fa
    fa.fa_paged_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["seqlens"],
                       new_lens=st["new_lens"], w=st["w"], weights=st["weights"])
    return [st["k_pages"], st["v_pages"], st["weights"]]


def _own_decode(st):
    import io_aware_attention_fa2_gb300 as fa
    o, lse = fa.paged_attention(st["q"], st["k_pages"], st["v_pages"], st["table"], st["seqlens"],
                                scale=st["scale"], weights=st["weights"],
                                window_left=st["window"])
    return [o, lse, st["weights"]]


def _own_evict(st):
    import io_aware_attention_fa2_gb300 as fa
    kept, lens = fa.paged_evict(st["k_pages"], st["v_pages"], st["weights"], st["table"],
                                st["seqlens"], st["out_table"], st["budget"], st["recent"])
    return [kept, lens, st["k_pages"], st["v_pages"], st["weights"]]


_own = dict(key_weights=_own_key_weights, append=_own_append, decode=_own_decode,
            evict=_own_evict)


# --------------------------------------------------------------------------- the plain forms
def _plain_key_weights(st):
    B, N, Hq, d = st["q"].shape
    Hkv = st["Hkv"]
    q = st["q"].float().view(B, N, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 3, 1)[:, :, None]
    p = torch.matmul(q, k)                                       # [B, Hkv, G, query, key]
    p.mul_(st["scale"]).sub_(st["lse"].view(B, Hkv, Hq // Hkv, N, 1)).exp_()
    i = torch.arange(N, device=DEV)
    n = (st["seqlens"] if st["seqlens"] is not None
         else torch.full((B,), N, dtype=torch.int32, device=DEV))
    see = (i[None, None, :] < n[:, None, None]) & (i[None, :, None] < n[:, None, None])
    if st["causal"]:
        see = see & (i[None, :] <= i[:, None])
    if st["window"] >= 0:
        see = see & (i[None, :] >= i[:, None] - st["window"])
    return p.masked_fill_(~see[:, None, None], 0.0).sum(dim=(2, 3))


def _slots(st, t):
    """Physical page and row of tokens t [B, n] of their sequences."""
    page = st["page"]
    col = (t // page).clamp(0, st["table"].shape[1] - 1)
    return st["table"].gather(1, col).long().clamp(min=0), t % page


def _plain_append(st):
    B, N = st["k"].shape[:2]
    i = torch.arange(N, device=DEV)
    new = i[None, :] < st["new_lens"][:, None]
    t = (st["seqlens"] - st["new_lens"])[:, None] + i[None, :]
    where, row = _slots(st, t)
    where, row = where[new], row[new]
    st["k_pages"][where, row] = st["k"][new]
    st["v_pages"][where, row] = st["v"][new]
    if st["weights"] is not None:
        st["weights"][where, :, row] = st["w"].transpose(1, 2)[new]
    return [st["k_pages"], st["v_pages"], st["weights"]]


def _plain_decode(st):
    B, Hq, d = st["q"].shape
    Hkv, page, table = st["Hkv"], st["page"], st["table"].long().clamp(min=0)
    n = table.shape[1] * page
    t = torch.arange(n, device=DEV)
    see = t[None, :] < st["seqlens"][:, None]
    if st["window"] >= 0:
        see = see & (t[None, :] >= st["seqlens"][:, None] - 1 - st["window"])
    q = st["q"].float().view(B, Hkv, Hq // Hkv, d)
    k = st["k_pages"][table].view(B, n, Hkv, d).permute(0, 2, 3, 1).float()
    s = torch.matmul(q, k) * st["scale"]                          # [B, Hkv, G, key]
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    p = torch.where(l > 0, p / l, torch.zeros_like(p))
    v = st["v_pages"][table].view(B, n, Hkv, d).permute(0, 2, 1, 3).float()
    v = torch.where(see[:, None, :, None], v, torch.zeros((), device=DEV))
    o = torch.matmul(p, v).view(B, Hq, d).to(st["q"].dtype)
    lse = (m + torch.log(l)).view(B, Hq)
    if st["weights"] is not None:
        where, row = _slots(st, t[None, :].expand(B, n))
        st["weights"][where[see], :, row[see]] += p.sum(dim=2).transpose(1, 2)[see]
    return [o, lse, st["weights"]]


def _plain_evict(st):
    B, Hkv, budget, page = st["B"], st["Hkv"], st["budget"], st["page"]
    width = st["table"].shape[1] * page
    t = torch.arange(width, device=DEV)
    n = st["seqlens"][:, None]
    where, row = _slots(st, t[None, :].expand(B, width))
    w = st["weights"][where, :, row].transpose(1, 2)              # [B, Hkv, token]
    w = torch.where((t >= n - st["recent"])[:, None], math.inf, w)
    w = torch.where((t >= n)[:, None], -math.inf, w)
    top = torch.sort(w, dim=-1, descending=True, stable=True).indices[:, :, :budget]
    kept = torch.sort(torch.where(top < n[:, None], top, width), dim=-1).values
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[2]), value=width)
    b, h, i = torch.nonzero(kept < width, as_tuple=True)
    src = kept[b, h, i]
    from_page, from_row = st["table"][b, src // page].long(), src % page
    to_page, to_row = st["out_table"][b, i // page].long(), i % page
    for pool in (st["k_pages"], st["v_pages"]):
        pool[to_page, to_row, h] = pool[from_page, from_row, h]
    st["weights"][to_page, h, to_row] = st["weights"][from_page, h, from_row]
    kept = torch.where(kept < width, kept, -1).to(torch.int32)
    return [kept, st["seqlens"].clamp(max=budget), st["k_pages"], st["v_pages"], st["weights"]]


_plain = dict(key_weights=_plain_key_weights, append=_plain_append, decode=_plain_decode,
              evict=_plain_evict)


# --------------------------------------------------------------------------- work and exact values
def work(case):
    d, B, Hkv = case["d"], case["B"], case["Hkv"]
    if case["op"] == "key_weights":
        pairs = 0
        for n in _key_lens(case):
            a = case["window"] if case["window"] >= 0 else n
            c = 0 if case["causal"] else n                         # keys ahead of the query
            # sum over queries i of min(i, a) keys behind, itself, and min(n - 1 - i, c) ahead
            pairs += n + sum(m * (m + 1) // 2 + max(0, n - 1 - m) * m for m in
                             (min(a, n - 1), min(c, n - 1)))
        return {"flops": 2.0 * d * pairs * case["Hq"],
                "bytes": 2.0 * B * case["N"] * d * (case["Hq"] + Hkv)
                + 4.0 * B * case["N"] * (case["Hq"] + Hkv)}
    if case["op"] == "append":
        new = sum(_lens(case, case["N"], 1))
        return {"flops": 0.0, "bytes": new * Hkv * (2 * 2 * 2 * d + (8 if case["weights"] else 0))}
    if case["op"] == "decode":
        seen = sum(min(n, case["window"] + 1) if case["window"] >= 0 else n
                   for n in _lens(case, case["len"]))
        return {"flops": 4.0 * seen * case["Hq"] * d,
                "bytes": seen * Hkv * (2.0 * 2 * d + (8 if case["weights"] else 0))
                + B * case["Hq"] * (4.0 * d + 4)}
    seen = sum(_lens(case, case["len"]))
    kept = sum(min(n, case["budget"]) for n in _lens(case, case["len"]))
    return {"flops": 0.0, "bytes": Hkv * (4.0 * seen + kept * (2 * 4 * d + 2 * 4 + 4))}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact[case["op"]](case, st)


def _exact_key_weights(case, st):
    """Head by head, from the definition."""
    Hq, Hkv, N = case["Hq"], case["Hkv"], case["N"]
    w = torch.zeros((case["B"], Hkv, N), dtype=torch.float64, device=DEV)
    i = torch.arange(N, device=DEV)
    for b, n in enumerate(_key_lens(case)):
        see = _visible(i, case, n)[:n, :n]
        for h in range(Hq):
            hk = h * Hkv // Hq
            s = torch.einsum("ic,jc->ij", st["q"][b, :n, h].double(), st["k"][b, :n, hk].double())
            p = torch.exp(s * st["scale"] - st["lse"][b, h, :n, None].double())
            w[b, hk, :n] += torch.where(see, p, 0.0).sum(dim=0)
    return w


def _rows(st, b, n):
    """(page, row) of the first n tokens of sequence b."""
    page = st["page"]
    return (st["table"][b, :_pages(n, page)].long().repeat_interleave(page)[:n],
            torch.arange(n, device=DEV) % page)


def _exact_append(case, st):
    k, v = st["k_pages"].double(), st["v_pages"].double()
    w = None if st["weights"] is None else st["weights"].double()
    for b, end in enumerate(st["seqlens"].tolist()):
        n = end - case["start"]
        pg, row = (x[case["start"]:] for x in _rows(st, b, end))
        k[pg, row], v[pg, row] = st["k"][b, :n].double(), st["v"][b, :n].double()
        if w is not None:
            w[pg, :, row] = st["w"][b, :, :n].double().T
    return [k, v, w]


def _exact_decode(case, st):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    o = torch.zeros((case["B"], Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"], Hq), -math.inf, dtype=torch.float64, device=DEV)
    w = None if st["weights"] is None else st["weights"].double()
    for b, n in enumerate(st["seqlens"].tolist()):
        if n == 0:
            continue
        first = max(0, n - 1 - case["window"]) if case["window"] >= 0 else 0
        pg, row = (x[first:] for x in _rows(st, b, n))
        for h in range(Hq):
            hk = h * Hkv // Hq
            s = st["k_pages"][pg, row, hk].double() @ st["q"][b, h].double() * st["scale"]
            lse[b, h] = torch.logsumexp(s, dim=0)
            p = torch.exp(s - lse[b, h])
            o[b, h] = p @ st["v_pages"][pg, row, hk].double()
            if w is not None:
                w[pg, hk, row] += p
    return [o, lse, w]


def _exact_evict(case, st):
    """kept and the new lengths are whole numbers; the moved values are looked up one head at a
    time, all of them before the first is written."""
    k, v, w = (st[x].double() for x in ("k_pages", "v_pages", "weights"))
    old = [x.clone() for x in (k, v, w)]
    page = case["page"]
    for b, n in enumerate(st["seqlens"].tolist()):
        m = min(n, case["budget"])
        pg, row = _rows(st, b, n)
        to_pg = st["out_table"][b].long().repeat_interleave(page)[:m]
        to_row = torch.arange(m, device=DEV) % page
        fixed = min(n, case["recent"])
        for h in range(case["Hkv"]):
            value = old[2][pg[:n - fixed], h, row[:n - fixed]]
            # by weight from the heaviest, equal ones from the oldest: sorted by (-weight, place)
            best = torch.argsort(-value, stable=True)[:m - fixed]
            keep = torch.cat([best.sort().values, torch.arange(n - fixed, n, device=DEV)])
            k[to_pg, to_row, h] = old[0][pg[keep], row[keep], h]
            v[to_pg, to_row, h] = old[1][pg[keep], row[keep], h]
            w[to_pg, h, to_row] = old[2][pg[keep], h, row[keep]]
    return [None, None, k, v, w]


_exact = dict(key_weights=_exact_key_weights, append=_exact_append, decode=_exact_decode,
              evict=_exact_evict)
