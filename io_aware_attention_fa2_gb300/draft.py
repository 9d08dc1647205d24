"""Drafted tokens and branching sequences over the paged key-value cache: ctypes binding over
fa_paged_tree, fa_paged_accept, fa_paged_copy, fa_paged_fork and fa_paged_resize of
``include/fa.h`` (argument marshalling only, like ``paged``).

A step of speculative decoding, for a batch whose drafted tokens form trees (``parents`` int32
[B, T]: an earlier drafted token, or -1 for the context):

    room = paged_resize(pool, block_table, seqlens, seqlens + T, page_size)  # == seqlens + T
    fa_paged_append(k, v, k_pages, v_pages, block_table, room)
    o, lse = paged_tree_attention(q, k_pages, v_pages, block_table, room, parents=parents)
    # ... the model goes on; leaf int32 [B] is the last drafted token that it agrees with ...
    path, seqlens = paged_accept(k_pages, v_pages, block_table, room, leaf, parents)
    paged_resize(pool, block_table, room, seqlens, page_size)

A pool (``new_page_pool``) says which pages are free and how many tables hold each. Several
continuations of a sequence share its whole pages:

    forked = paged_fork(pool, block_table, seqlens, source, page_size)
    fa_paged_copy(k_pages, v_pages, forked.copy_src, forked.copy_dst, rows=forked.copy_rows)

with the copies made in the pages of every layer. Tensors, streams and ``device_error()`` as in
``paged``.
"""
from __future__ import annotations

import functools
from typing import NamedTuple

from .binding import _dtype_code, load_library
from .paged import (_bound, _cache, _call, _check, _count, _default_scale, _library, _ptr,
                    _stream_of, _workspace)


@functools.lru_cache(maxsize=256)
def paged_tree_workspace_size(B: int, T: int, Hq: int, Hkv: int, d: int, page_size: int,
                              max_pages: int) -> int:
    """Bytes of workspace fa_paged_tree needs."""
    return int(load_library().fa_paged_tree_workspace_size(B, T, Hq, Hkv, d, page_size, max_pages))


def fa_paged_tree(q, k_pages, v_pages, block_table, seqlens, o, lse, scale: float, parents=None,
                  new_lens=None, window_left: int = -1, workspace=None, stream=None) -> None:
    """Enqueue the attention of drafted tokens: q, o [B, T, Hq, d], lse float32 [B, Hq, T]. The
    last new_lens[b] (int32 [B]; None: all T) tokens of sequence b are the drafted ones, which
    seqlens[b] counts already; token i sees the context, its ancestors by ``parents`` (int32
    [B, T]; None: a chain) and itself, with ``window_left`` >= 0 only those at most that many
    positions before it. ``workspace``: a CUDA tensor of at least ``paged_tree_workspace_size``
    bytes (16-byte aligned), or None to let PyTorch allocate one."""
    _tree(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, parents, new_lens, window_left,
          workspace, stream)


def _tree(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, parents, new_lens, window_left,
          workspace, stream):
    """fa_paged_tree; outputs that are None are allocated. Returns o, lse."""
    import torch
    device, dtype, B, Hkv, d, page_size, num_pages, max_pages = _cache(
        k_pages, v_pages, None, block_table, seqlens)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d]")
    T, Hq = q.shape[1], q.shape[2]
    _check("q", q, (B, T, Hq, d), dtype, device)
    if parents is not None:
        _check("parents", parents, (B, T), torch.int32, device)
    if new_lens is not None:
        _check("new_lens", new_lens, (B,), torch.int32, device)
    if o is None or lse is None:
        with _stream_of(stream, device):
            if o is None:
                o = torch.empty_like(q)
            if lse is None:
                lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
    _check("o", o, (B, T, Hq, d), dtype, device)
    _check("lse", lse, (B, Hq, T), torch.float32, device)
    need = 0 if workspace is not None else paged_tree_workspace_size(
        B, T, Hq, Hkv, d, page_size, max_pages)
    keep, ws, ws_bytes = _workspace(need, workspace, device, stream)
    _call("fa_paged_tree", _library().fa_paged_tree, device, stream, (
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
        seqlens.data_ptr(), _ptr(parents), _ptr(new_lens), o.data_ptr(), lse.data_ptr(), B, T, Hq,
        Hkv, d, page_size, num_pages, max_pages, _bound(window_left), float(scale), _dtype_code(q),
        ws, ws_bytes))
    return o, lse


def paged_tree_attention(q, k_pages, v_pages, block_table, seqlens, parents=None, new_lens=None,
                         scale: float | None = None, window_left: int = -1, out=None, lse=None,
                         workspace=None, stream=None):
    """O, LSE = attention of the drafted tokens of every sequence over a paged cache (see
    ``fa_paged_tree``; outputs are allocated here unless given). ``scale`` defaults to 1/sqrt(d)
    rounded to fp32."""
    if scale is None:
        scale = _default_scale(q.shape[-1])
    return _tree(q, k_pages, v_pages, block_table, seqlens, out, lse, scale, parents, new_lens,
                 window_left, workspace, stream)


def fa_paged_accept(k_pages, v_pages, block_table, seqlens, leaf, path, new_seqlens, parents=None,
                    new_lens=None, weights=None, stream=None) -> None:
    """Enqueue the move of the drafted tokens that stay behind the context: leaf[b] (int32 [B];
    -1: none) and its ancestors. path int32 [B, T] gets them in their order (-1 behind the last),
    new_seqlens int32 [B] the new lengths; ``weights`` of a cache that keeps them move, too."""
    import torch
    device, dtype, B, Hkv, d, page_size, num_pages, max_pages = _cache(
        k_pages, v_pages, weights, block_table, seqlens)
    if path.dim() != 2:
        raise ValueError("path must be [B, T]")
    T = _count("T", path.shape[1])
    _check("path", path, (B, T), torch.int32, device)
    _check("leaf", leaf, (B,), torch.int32, device)
    _check("new_seqlens", new_seqlens, (B,), torch.int32, device)
    if parents is not None:
        _check("parents", parents, (B, T), torch.int32, device)
    if new_lens is not None:
        _check("new_lens", new_lens, (B,), torch.int32, device)
    _call("fa_paged_accept", _library().fa_paged_accept, device, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), _ptr(weights), block_table.data_ptr(),
        seqlens.data_ptr(), _ptr(parents), leaf.data_ptr(), _ptr(new_lens), path.data_ptr(),
        new_seqlens.data_ptr(), B, T, Hkv, d, page_size, num_pages, max_pages,
        _dtype_code(k_pages)))


def paged_accept(k_pages, v_pages, block_table, seqlens, leaf, parents, new_lens=None,
                 weights=None, stream=None):
    """path, new_seqlens = the drafted tokens that stay, moved behind the context (see
    ``fa_paged_accept``)."""
    import torch
    if parents.dim() != 2:
        raise ValueError("parents must be [B, T]")
    with _stream_of(stream, k_pages.device):
        path = torch.empty_like(parents)
        new_seqlens = torch.empty_like(seqlens)
    fa_paged_accept(k_pages, v_pages, block_table, seqlens, leaf, path, new_seqlens, parents,
                    new_lens, weights, stream)
    return path, new_seqlens


def fa_paged_copy(k_pages, v_pages, src, dst, rows=None, weights=None, stream=None) -> None:
    """Enqueue copies of pages: the first rows[m] rows (int32 [M]; None: all) of page src[m] to page
    dst[m] (int32 [M]; both negative: no copy), keys, values and ``weights`` of a cache that keeps
    them."""
    import torch
    from .paged import _first
    device, dtype = _first("k_pages", k_pages, 4)
    num_pages, page_size, Hkv, d = k_pages.shape
    _check("v_pages", v_pages, k_pages.shape, dtype, device)
    if weights is not None:
        _check("weights", weights, (num_pages, Hkv, page_size), torch.float32, device)
    if src.dim() != 1:
        raise ValueError("src must be [M]")
    M = _count("M", src.shape[0])
    _check("src", src, (M,), torch.int32, device)
    _check("dst", dst, (M,), torch.int32, device)
    if rows is not None:
        _check("rows", rows, (M,), torch.int32, device)
    _call("fa_paged_copy", _library().fa_paged_copy, device, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), _ptr(weights), src.data_ptr(), dst.data_ptr(),
        _ptr(rows), M, Hkv, d, page_size, num_pages, _dtype_code(k_pages)))


class PagePool(NamedTuple):
    """A pool's books: refs int32 [num_pages], how many tables hold a page; free_pages int32
    [num_pages], whose first num_free[0] entries are the free pages, the last taken first; num_free
    int32 [1]."""
    refs: "torch.Tensor"        # noqa: F821
    free_pages: "torch.Tensor"  # noqa: F821
    num_free: "torch.Tensor"    # noqa: F821


def new_page_pool(num_pages: int, device="cuda") -> PagePool:
    """The books of a pool whose pages are all free; page 0 is taken first."""
    import torch
    if not 1 <= _count("num_pages", num_pages):
        raise ValueError("num_pages must be at least 1")
    return PagePool(torch.zeros(num_pages, dtype=torch.int32, device=device),
                    torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
                    torch.full((1,), num_pages, dtype=torch.int32, device=device))


def _tables(pool, block_table):
    """Checks a pool and a block table: (device, B, max_pages, num_pages)."""
    import torch
    if block_table.dim() != 2 or not block_table.is_cuda or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous 2-D CUDA tensor")
    device, (B, max_pages) = block_table.device, block_table.shape
    num_pages = pool.refs.numel()
    _count("num_pages", num_pages)
    _count("B", B)
    _count("max_pages", max_pages)
    _check("block_table", block_table, (B, max_pages), torch.int32, device)
    _check("refs", pool.refs, (num_pages,), torch.int32, device)
    _check("free_pages", pool.free_pages, (num_pages,), torch.int32, device)
    _check("num_free", pool.num_free, (1,), torch.int32, device)
    return device, B, max_pages, num_pages


class Forked(NamedTuple):
    """What a fork gives: the new sequences' table int32 [C, max_pages] and lengths int32 [C] (-1:
    the pool was empty), and the copies to make in every layer's pages (``fa_paged_copy``)."""
    block_table: "torch.Tensor"  # noqa: F821
    seqlens: "torch.Tensor"      # noqa: F821
    copy_src: "torch.Tensor"     # noqa: F821
    copy_dst: "torch.Tensor"     # noqa: F821
    copy_rows: "torch.Tensor"    # noqa: F821


def fa_paged_fork(pool, block_table, seqlens, source, out: Forked, page_size: int,
                  stream=None) -> None:
    """Enqueue a fork: sequence c of ``out`` continues sequence source[c] (int32 [C]; -1: empty),
    with its whole pages shared and its last one, where it is filled in part, from the pool."""
    import torch
    device, B, max_pages, num_pages = _tables(pool, block_table)
    _check("seqlens", seqlens, (B,), torch.int32, device)
    if source.dim() != 1:
        raise ValueError("source must be [C]")
    C = _count("C", source.shape[0])
    _check("source", source, (C,), torch.int32, device)
    _check("out.block_table", out.block_table, (C, max_pages), torch.int32, device)
    for name in ("seqlens", "copy_src", "copy_dst", "copy_rows"):
        _check("out." + name, getattr(out, name), (C,), torch.int32, device)
    _call("fa_paged_fork", _library().fa_paged_fork, device, stream, (
        block_table.data_ptr(), seqlens.data_ptr(), source.data_ptr(), pool.refs.data_ptr(),
        pool.free_pages.data_ptr(), pool.num_free.data_ptr(), out.block_table.data_ptr(),
        out.seqlens.data_ptr(), out.copy_src.data_ptr(), out.copy_dst.data_ptr(),
        out.copy_rows.data_ptr(), B, C, _count("page_size", page_size), num_pages, max_pages))


def paged_fork(pool, block_table, seqlens, source, page_size: int, stream=None) -> Forked:
    """New sequences that continue others (see ``fa_paged_fork``), in tables of their own."""
    import torch
    if block_table.dim() != 2 or source.dim() != 1:
        raise ValueError("block_table must be [B, max_pages] and source [C]")
    C = source.shape[0]
    with _stream_of(stream, block_table.device):
        # one allocation for the lists: the call is a few microseconds long
        lists = torch.empty((4, C), dtype=torch.int32, device=block_table.device)
        table = torch.empty((C, block_table.shape[1]), dtype=torch.int32,
                            device=block_table.device)
    out = Forked(table, *lists.unbind(0))
    fa_paged_fork(pool, block_table, seqlens, source, out, page_size, stream)
    return out


def fa_paged_resize(pool, block_table, old_lens, new_lens, granted, page_size: int,
                    stream=None) -> None:
    """Enqueue a change of lengths: sequence b has pages for old_lens[b] tokens and gets those for
    new_lens[b], given back to the pool or taken from it, in its row of block_table. granted
    int32 [B] gets new_lens[b], or old_lens[b] where the pool did not suffice."""
    import torch
    device, B, max_pages, num_pages = _tables(pool, block_table)
    for name, t in (("old_lens", old_lens), ("new_lens", new_lens), ("granted", granted)):
        _check(name, t, (B,), torch.int32, device)
    _call("fa_paged_resize", _library().fa_paged_resize, device, stream, (
        block_table.data_ptr(), old_lens.data_ptr(), new_lens.data_ptr(), granted.data_ptr(),
        pool.refs.data_ptr(), pool.free_pages.data_ptr(), pool.num_free.data_ptr(), B,
        _count("page_size", page_size), num_pages, max_pages))


def paged_resize(pool, block_table, old_lens, new_lens, page_size: int, stream=None):
    """granted int32 [B]: the lengths that the tables have pages for after ``fa_paged_resize``."""
    import torch
    with _stream_of(stream, block_table.device):
        granted = torch.empty_like(old_lens)
    fa_paged_resize(pool, block_table, old_lens, new_lens, granted, page_size, stream)
    return granted
