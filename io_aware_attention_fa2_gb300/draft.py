"""Drafted tokens and branching sequences over the paged key-value cache: ctypes binding over
fa_paged_tree, fa_paged_accept, fa_paged_copy, fa_paged_fork and fa_paged_resize of
``include/fa.h`` (argument marshalling only, like ``paged``).

A step of speculative decoding, for a batch whose drafted tokens form trees (``parents`` int32
[B, T]: an earlier drafted token, or -1 for the context):

    room = paged_resize(pool, block_table, seqlens, seqlens + T, page_size)
    drafted = room - seqlens            # T, or 0 for a sequence that the pool had no pages for
    fa_paged_append(k, v, k_pages, v_pages, block_table, room, new_lens=drafted)
    o, lse = paged_tree_attention(q, k_pages, v_pages, block_table, room, parents=parents,
                                  new_lens=drafted)
    # ... the model goes on; leaf int32 [B] is the last drafted token that it agrees with, or -1 ...
    path, seqlens = paged_accept(k_pages, v_pages, block_table, room, leaf, parents,
                                 new_lens=drafted)
    paged_resize(pool, block_table, room, seqlens, page_size)

Drafts that are chains need no ``parents`` (``paged_accept`` then takes their width as ``T``), and
their masks cost less. Nothing here adds to the weights of a cache that keeps them: accepted tokens
bring theirs along, their queries' attention to the others is not counted.

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

from .binding import FA_OK, FaError, _dtype_code, load_library
from .paged import (_NO_CONTEXT, _bound, _call, _check, _count, _default_scale, _first, _library, _ptr,
                    _stream_of, _workspace)

_INT_MAX = 2 ** 31 - 1


@functools.lru_cache(maxsize=None)
def _torch():
    """torch and what the calls below take of it: a few microseconds of GPU work stand against
    every name looked up."""
    import torch
    return (torch, torch.int32, torch.float32, torch.empty_like, torch._C._cuda_getDevice,
            torch._C._cuda_getCurrentRawStream)


def _fits(name, t, shape, dtype, device):
    """``_check`` with the device's number, which is quicker to ask for than the device."""
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != device
            or not t.is_contiguous()):
        _check(name, t, shape, dtype, _torch()[0].device("cuda", device))


def _pages(k_pages, v_pages):
    """Checks a cache's pages: (device, dtype, num_pages, page_size, Hkv, d)."""
    if k_pages.dim() != 4 or not k_pages.is_cuda or not k_pages.is_contiguous():
        _first("k_pages", k_pages, 4)
    device, dtype, shape = k_pages.get_device(), k_pages.dtype, k_pages.shape
    _fits("v_pages", v_pages, shape, dtype, device)
    return (device, dtype, *shape)


def _sequences(block_table, device):
    """Checks a block table: (B, max_pages)."""
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = shape
    if B > _INT_MAX or max_pages > _INT_MAX:
        raise ValueError("block_table is too large: %s" % list(shape))
    _fits("block_table", block_table, shape, _torch()[1], device)
    return B, max_pages


def _enqueue(where, fn, device, stream, args):
    """fn(*args, stream) on device number `device`."""
    torch, _, _, _, current, raw_stream = _torch()
    if stream is None and current() == device:
        rc = fn(*args, raw_stream(device) or None)
        if rc != FA_OK:
            raise FaError(rc, where)
    else:
        _call(where, fn, torch.device("cuda", device), stream, args)


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
    torch, int32, float32, empty_like, _, _ = _torch()
    device, dtype, num_pages, page_size, Hkv, d = _pages(k_pages, v_pages)
    B, max_pages = _sequences(block_table, device)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, d]")
    _, T, Hq, _ = shape = q.shape
    _fits("q", q, (B, T, Hq, d), dtype, device)
    _fits("seqlens", seqlens, (B,), int32, device)
    if parents is not None:
        _fits("parents", parents, (B, T), int32, device)
    if new_lens is not None:
        _fits("new_lens", new_lens, (B,), int32, device)
    if o is not None:
        _fits("o", o, shape, dtype, device)
    if lse is not None:
        _fits("lse", lse, (B, Hq, T), float32, device)
    if o is None or lse is None:
        with _NO_CONTEXT if stream is None else _stream_of(stream, q.device):
            if o is None:
                o = empty_like(q)
            if lse is None:
                lse = torch.empty((B, Hq, T), dtype=float32, device=q.device)
    need = 0 if workspace is not None else paged_tree_workspace_size(
        B, T, Hq, Hkv, d, page_size, max_pages)
    keep, ws, ws_bytes = ((None, None, 0) if need == 0 and workspace is None else
                          _workspace(need, workspace, q.device, stream))
    _enqueue("fa_paged_tree", _library().fa_paged_tree, device, stream, (
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
        seqlens.data_ptr(), _ptr(parents), _ptr(new_lens), o.data_ptr(), lse.data_ptr(), B, T, Hq,
        Hkv, d, page_size, num_pages, max_pages, _bound(window_left), float(scale), _dtype_code(q), ws,
        ws_bytes))
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
    if path.dim() != 2:
        raise ValueError("path must be [B, T]")
    _accept(k_pages, v_pages, block_table, seqlens, leaf, path, new_seqlens, parents, new_lens,
            weights, stream)


def _accept(k_pages, v_pages, block_table, seqlens, leaf, path, new_seqlens, parents, new_lens,
            weights, stream, T=None):
    """fa_paged_accept; outputs that are None are allocated. Returns path, new_seqlens."""
    torch, int32, float32, empty_like, _, _ = _torch()
    if T is None:
        T = (parents if path is None else path).shape[1]
    T = _count("T", T)
    device, dtype, num_pages, page_size, Hkv, d = _pages(k_pages, v_pages)
    B, max_pages = _sequences(block_table, device)
    _fits("seqlens", seqlens, (B,), int32, device)
    _fits("leaf", leaf, (B,), int32, device)
    if weights is not None:
        _fits("weights", weights, (num_pages, Hkv, page_size), float32, device)
    if parents is not None:
        _fits("parents", parents, (B, T), int32, device)
    if new_lens is not None:
        _fits("new_lens", new_lens, (B,), int32, device)
    if path is None:
        with _NO_CONTEXT if stream is None else _stream_of(stream, k_pages.device):
            path = (torch.empty((B, max(T, 0)), dtype=int32, device=k_pages.device)
                    if parents is None else empty_like(parents))
            new_seqlens = empty_like(seqlens)
    else:
        _fits("path", path, (B, T), int32, device)
        _fits("new_seqlens", new_seqlens, (B,), int32, device)
    _enqueue("fa_paged_accept", _library().fa_paged_accept, device, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), _ptr(weights), block_table.data_ptr(),
        seqlens.data_ptr(), _ptr(parents), leaf.data_ptr(), _ptr(new_lens), path.data_ptr(),
        new_seqlens.data_ptr(), B, T, Hkv, d, page_size, num_pages, max_pages,
        _dtype_code(k_pages)))
    return path, new_seqlens


def paged_accept(k_pages, v_pages, block_table, seqlens, leaf, parents=None, new_lens=None,
                 weights=None, stream=None, T: int | None = None):
    """path, new_seqlens = the drafted tokens that stay, moved behind the context (see
    ``fa_paged_accept``). ``T``: the width of the draft, for chains without ``parents``."""
    if parents is None:
        if T is None:
            raise ValueError("T has to be given where parents are not")
    elif parents.dim() != 2 or (T is not None and parents.shape[1] != T):
        raise ValueError("parents must be [B, T]")
    return _accept(k_pages, v_pages, block_table, seqlens, leaf, None, None, parents, new_lens,
                   weights, stream, T)


def fa_paged_copy(k_pages, v_pages, src, dst, rows=None, weights=None, stream=None) -> None:
    """Enqueue copies of pages: the first rows[m] rows (int32 [M]; None: all) of page src[m] to page
    dst[m] (int32 [M]; both negative: no copy), keys, values and ``weights`` of a cache that keeps
    them."""
    _, int32, float32, _, _, _ = _torch()
    device, dtype, num_pages, page_size, Hkv, d = _pages(k_pages, v_pages)
    if weights is not None:
        _fits("weights", weights, (num_pages, Hkv, page_size), float32, device)
    if src.dim() != 1:
        raise ValueError("src must be [M]")
    M = _count("M", src.shape[0])
    _fits("src", src, (M,), int32, device)
    _fits("dst", dst, (M,), int32, device)
    if rows is not None:
        _fits("rows", rows, (M,), int32, device)
    _enqueue("fa_paged_copy", _library().fa_paged_copy, device, stream, (
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
    if block_table.dim() != 2 or not block_table.is_cuda or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous 2-D CUDA tensor")
    int32, device = _torch()[1], block_table.get_device()
    B, max_pages = _sequences(block_table, device)
    refs, free_pages, num_free = pool
    shape = refs.shape
    if len(shape) != 1 or shape[0] > _INT_MAX:
        raise ValueError("refs must be [num_pages]")
    _fits("refs", refs, shape, int32, device)
    _fits("free_pages", free_pages, shape, int32, device)
    _fits("num_free", num_free, (1,), int32, device)
    return device, B, max_pages, shape[0]


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
    _fork(pool, block_table, seqlens, source, out, page_size, stream)


def _fork(pool, block_table, seqlens, source, out, page_size, stream):
    """fa_paged_fork; an `out` that is None is allocated. Returns it."""
    torch, int32, _, empty_like, _, _ = _torch()
    device, B, max_pages, num_pages = _tables(pool, block_table)
    refs, free_pages, num_free = pool
    _fits("seqlens", seqlens, (B,), int32, device)
    if source.dim() != 1:
        raise ValueError("source must be [C]")
    shape = source.shape
    C = _count("C", shape[0])
    _fits("source", source, shape, int32, device)
    page_size = _count("page_size", page_size)
    if out is None:
        with _NO_CONTEXT if stream is None else _stream_of(stream, block_table.device):
            # (four allocations cost less than views of one)
            out = Forked(torch.empty((C, max_pages), dtype=int32, device=source.device),
                         empty_like(source), empty_like(source), empty_like(source),
                         empty_like(source))
        table, lens, src, dst, rows = out
    else:
        table, lens, src, dst, rows = out
        _fits("out.block_table", table, (C, max_pages), int32, device)
        _fits("out.seqlens", lens, shape, int32, device)
        _fits("out.copy_src", src, shape, int32, device)
        _fits("out.copy_dst", dst, shape, int32, device)
        _fits("out.copy_rows", rows, shape, int32, device)
    _enqueue("fa_paged_fork", _library().fa_paged_fork, device, stream, (
        block_table.data_ptr(), seqlens.data_ptr(), source.data_ptr(), refs.data_ptr(),
        free_pages.data_ptr(), num_free.data_ptr(), table.data_ptr(), lens.data_ptr(),
        src.data_ptr(), dst.data_ptr(), rows.data_ptr(), B, C, page_size, num_pages, max_pages))
    return out


def paged_fork(pool, block_table, seqlens, source, page_size: int, stream=None) -> Forked:
    """New sequences that continue others (see ``fa_paged_fork``), in tables of their own."""
    return _fork(pool, block_table, seqlens, source, None, page_size, stream)


def fa_paged_resize(pool, block_table, old_lens, new_lens, granted, page_size: int,
                    stream=None) -> None:
    """Enqueue a change of lengths: sequence b has pages for old_lens[b] tokens and gets those for
    new_lens[b], given back to the pool or taken from it, in its row of block_table. granted
    int32 [B] gets new_lens[b], or old_lens[b] where the pool did not suffice."""
    _resize(pool, block_table, old_lens, new_lens, granted, page_size, stream)


def _resize(pool, block_table, old_lens, new_lens, granted, page_size, stream):
    """fa_paged_resize; a `granted` that is None is allocated. Returns it."""
    _, int32, _, empty_like, _, _ = _torch()
    device, B, max_pages, num_pages = _tables(pool, block_table)
    refs, free_pages, num_free = pool
    shape = (B,)
    _fits("old_lens", old_lens, shape, int32, device)
    _fits("new_lens", new_lens, shape, int32, device)
    page_size = _count("page_size", page_size)
    if granted is None:
        with _NO_CONTEXT if stream is None else _stream_of(stream, block_table.device):
            granted = empty_like(old_lens)
    else:
        _fits("granted", granted, shape, int32, device)
    _enqueue("fa_paged_resize", _library().fa_paged_resize, device, stream, (
        block_table.data_ptr(), old_lens.data_ptr(), new_lens.data_ptr(), granted.data_ptr(),
        refs.data_ptr(), free_pages.data_ptr(), num_free.data_ptr(), B, page_size, num_pages,
        max_pages))
    return granted


def paged_resize(pool, block_table, old_lens, new_lens, page_size: int, stream=None):
    """granted int32 [B]: the lengths that the tables have pages for after ``fa_paged_resize``."""
    return _resize(pool, block_table, old_lens, new_lens, None, page_size, stream)
