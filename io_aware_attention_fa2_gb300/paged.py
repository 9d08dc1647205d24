"""The paged key-value cache: ctypes binding over the fa_key_weights and fa_paged_* entry points
of ``include/fa.h`` (argument marshalling only, like ``binding``).

A cache is two tensors ``k_pages``, ``v_pages`` [num_pages, page_size, Hkv, d] and, when it is to
be kept within a budget, ``weights`` float32 [num_pages, Hkv, page_size]: the attention weight
every token has received so far. ``block_table`` int32 [B, max_pages] and ``seqlens`` int32 [B]
say which rows belong to which sequence. The life of a sequence, with G = Hq // Hkv query heads to
a key head (the forward wants keys and values for every query head):

    o, lse = attention_forward(q, k.repeat_interleave(G, 2), v.repeat_interleave(G, 2), causal=True)
    w = key_weights(q, k, lse, causal=True)
    fa_paged_append(k, v, k_pages, v_pages, block_table, seqlens, w=w, weights=weights)
    for each new token:                                        # seqlens counts it already
        fa_paged_append(k1, v1, k_pages, v_pages, block_table, seqlens, weights=weights)
        o1, lse1 = paged_attention(q1, k_pages, v_pages, block_table, seqlens, weights=weights)
    kept, seqlens = paged_evict(k_pages, v_pages, weights, block_table, seqlens, free_pages,
                                budget, recent)
    block_table, free_pages = free_pages, block_table          # where the kept tokens are now

Every tensor is a contiguous CUDA tensor of one device; calls run on that device and, unless a
``stream`` is given, on its current stream. A block-table entry or length that names a token
outside the cache is found on the device: ``device_error()`` then returns ``FA_ERR_PAGE``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

from . import binding
from .binding import FA_OK, FaError, _dtype_code, load_library

_NO_CONTEXT = contextlib.nullcontext()
_INT_MAX = 2 ** 31 - 1   # ctypes would pass the low 32 bits of a larger number


def _library():
    return binding._lib or load_library()


def _check(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor %s on %s" % (
            name, str(dtype).replace("torch.", ""), list(shape), device))


def _count(name, n):
    """A number that the library takes as an int."""
    n = int(n)
    if not -_INT_MAX <= n <= _INT_MAX:
        raise ValueError("%s is out of range: %d" % (name, n))
    return n


def _bound(n):
    """A window bound: any negative number is none, and one past every length is as good."""
    n = int(n)
    return -1 if n < 0 else min(n, _INT_MAX)


def _first(name, t, dims):
    """The tensor that sets the call's device and dtype."""
    if t.dim() != dims or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-D CUDA tensor" % (name, dims))
    return t.device, t.dtype


def _call(where, fn, device, stream, args):
    """fn(*args, stream) on the tensors' device (the library works on the current one)."""
    import torch
    if torch._C._cuda_getDevice() != device.index:
        with torch.cuda.device(device):
            return _call(where, fn, device, stream, args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        stream = getattr(stream, "cuda_stream", stream)
    rc = fn(*args, stream or None)
    if rc != FA_OK:
        raise FaError(rc, where)


def _stream_of(stream, device):
    """Allocations inside belong to the call's stream."""
    import torch
    if stream is None:
        return _NO_CONTEXT
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _workspace(need, workspace, device, stream):
    """(tensor, address, bytes) of a workspace: the caller's, or one of `need` bytes that PyTorch
    allocates for the call's stream, so that it is reused only by later work there."""
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on %s" % device)
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    import torch
    if stream is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        with _stream_of(stream, device):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, workspace.data_ptr(), need


def _cache(k_pages, v_pages, weights, block_table, seqlens):
    """Checks a cache's tensors: (device, dtype, B, Hkv, d, page_size, num_pages, max_pages)."""
    import torch
    device, dtype = _first("k_pages", k_pages, 4)
    shape = k_pages.shape
    num_pages, page_size, Hkv, d = shape
    _check("v_pages", v_pages, shape, dtype, device)
    table = block_table.shape
    if len(table) != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = table
    if B > _INT_MAX or max_pages > _INT_MAX:
        raise ValueError("block_table is too large: %s" % list(table))
    _check("block_table", block_table, table, torch.int32, device)
    _check("seqlens", seqlens, (B,), torch.int32, device)
    if weights is not None:
        _check("weights", weights, (num_pages, Hkv, page_size), torch.float32, device)
    return device, dtype, B, Hkv, d, page_size, num_pages, max_pages


def _ptr(t):
    return None if t is None else t.data_ptr()


def _default_scale(d):
    return ctypes.c_float(1.0 / math.sqrt(d)).value


@functools.lru_cache(maxsize=256)
def key_weights_workspace_size(B: int, Hq: int, Hkv: int, N: int) -> int:
    """Bytes of workspace fa_key_weights needs (0 unless query heads share key heads)."""
    return int(load_library().fa_key_weights_workspace_size(B, Hq, Hkv, N))


def fa_key_weights(q, k, lse, w, causal: bool, scale: float, workspace=None, stream=None,
                   window=(-1, -1), seqlens_k=None) -> None:
    """Enqueue the weights that the keys of a prompt received: w [B, Hkv, N] float32 from
    q [B, N, Hq, d], k [B, N, Hkv, d] and the forward's lse [B, Hq, N]. ``window`` and
    ``seqlens_k`` as in ``fa_fwd``; queries at or past seqlens_k[b] add nothing."""
    import torch
    device, dtype = _first("q", q, 4)
    B, N, Hq, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, N, Hkv, d]")
    Hkv = k.shape[2]
    _check("k", k, (B, N, Hkv, d), dtype, device)
    _check("lse", lse, (B, Hq, N), torch.float32, device)
    _check("w", w, (B, Hkv, N), torch.float32, device)
    if seqlens_k is not None:
        _check("seqlens_k", seqlens_k, (B,), torch.int32, device)
    left, right = (_bound(x) for x in window)
    keep, ws, ws_bytes = _workspace(key_weights_workspace_size(B, Hq, Hkv, N), workspace, device,
                                    stream)
    _call("fa_key_weights", _library().fa_key_weights, device, stream, (
        q.data_ptr(), k.data_ptr(), lse.data_ptr(), w.data_ptr(), B, Hq, Hkv, N, d,
        int(bool(causal)), left, right, _ptr(seqlens_k), float(scale), _dtype_code(q), ws,
        ws_bytes))


def key_weights(q, k, lse, causal: bool = False, scale: float | None = None, stream=None,
                window=(-1, -1), seqlens_k=None, out=None):
    """w [B, Hkv, N]: the attention weight every key of a prompt received from the queries (and
    query heads) that see it. ``lse`` is what ``attention_forward`` returned for the same q, k
    and masks (``seqlens_k`` may be on the host, as there); ``scale`` defaults to 1/sqrt(d) rounded
    to fp32."""
    import torch
    if scale is None:
        scale = _default_scale(q.shape[-1])
    with _stream_of(stream, q.device):
        if out is None:
            out = torch.empty((q.shape[0], k.shape[2], q.shape[1]), dtype=torch.float32,
                              device=q.device)
        if seqlens_k is not None:
            seqlens_k = seqlens_k.to(q.device, torch.int32)
    fa_key_weights(q, k, lse, out, causal, scale, None, stream, window, seqlens_k)
    return out


def fa_paged_append(k, v, k_pages, v_pages, block_table, seqlens, new_lens=None, w=None,
                    weights=None, stream=None) -> None:
    """Enqueue the writing of new tokens into the pages: k, v [B, N, Hkv, d], of which the first
    new_lens[b] (int32 [B]; None: all N) become the last tokens of sequence b, whose seqlens[b]
    counts them already. With ``weights`` the new tokens get the weights ``w`` [B, Hkv, N]
    (None: 0)."""
    import torch
    device, dtype, B, Hkv, d, page_size, num_pages, max_pages = _cache(
        k_pages, v_pages, weights, block_table, seqlens)
    if k.dim() != 4:
        raise ValueError("k must be [B, N, Hkv, d]")
    N = k.shape[1]
    _check("k", k, (B, N, Hkv, d), dtype, device)
    _check("v", v, (B, N, Hkv, d), dtype, device)
    if new_lens is not None:
        _check("new_lens", new_lens, (B,), torch.int32, device)
    if w is not None:
        if weights is None:
            raise ValueError("w needs a cache with weights")
        _check("w", w, (B, Hkv, N), torch.float32, device)
    _call("fa_paged_append", _library().fa_paged_append, device, stream, (
        k.data_ptr(), v.data_ptr(), _ptr(w), k_pages.data_ptr(), v_pages.data_ptr(),
        _ptr(weights), block_table.data_ptr(), seqlens.data_ptr(), _ptr(new_lens), B, N, Hkv, d,
        page_size, num_pages, max_pages, _dtype_code(k)))


@functools.lru_cache(maxsize=256)
def paged_decode_workspace_size(B: int, Hq: int, Hkv: int, d: int, page_size: int,
                                max_pages: int, with_weights: bool = False) -> int:
    """Bytes of workspace fa_paged_decode needs."""
    return int(load_library().fa_paged_decode_workspace_size(B, Hq, Hkv, d, page_size, max_pages,
                                                             int(bool(with_weights))))


def fa_paged_decode(q, k_pages, v_pages, block_table, seqlens, o, lse, scale: float,
                    weights=None, window_left: int = -1, workspace=None, stream=None) -> None:
    """Enqueue the attention of one new token per sequence: q, o [B, Hq, d], lse float32
    [B, Hq]; with ``weights`` every visible token's probability (summed over the query heads of
    its key head) is added to them. ``window_left`` >= 0: only the last window_left + 1 tokens
    are visible. ``workspace``: a CUDA tensor of at least ``paged_decode_workspace_size`` bytes
    (16-byte aligned), or None to let PyTorch allocate one."""
    _decode(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, weights, window_left,
            workspace, stream)


def _decode(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, weights, window_left,
            workspace, stream):
    """fa_paged_decode; outputs that are None are allocated. Returns o, lse."""
    import torch
    device, dtype, B, Hkv, d, page_size, num_pages, max_pages = _cache(
        k_pages, v_pages, weights, block_table, seqlens)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    Hq = q.shape[1]
    _check("q", q, (B, Hq, d), dtype, device)
    if o is None or lse is None:
        with _stream_of(stream, device):
            if o is None:
                o = torch.empty_like(q)
            if lse is None:
                lse = torch.empty((B, Hq), dtype=torch.float32, device=device)
    _check("o", o, (B, Hq, d), dtype, device)
    _check("lse", lse, (B, Hq), torch.float32, device)
    need = 0 if workspace is not None else paged_decode_workspace_size(
        B, Hq, Hkv, d, page_size, max_pages, weights is not None)
    keep, ws, ws_bytes = _workspace(need, workspace, device, stream)
    _call("fa_paged_decode", _library().fa_paged_decode, device, stream, (
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(weights),
        block_table.data_ptr(), seqlens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, d,
        page_size, num_pages, max_pages, _bound(window_left), float(scale), _dtype_code(q), ws,
        ws_bytes))
    return o, lse


def paged_attention(q, k_pages, v_pages, block_table, seqlens, scale: float | None = None,
                    weights=None, window_left: int = -1, out=None, lse=None, workspace=None,
                    stream=None):
    """O, LSE = attention of one new token per sequence over a paged cache. The call a user makes
    for a decoding step (``fa_paged_decode`` with outputs allocated here unless given); ``scale``
    defaults to 1/sqrt(d) rounded to fp32."""
    if scale is None:
        scale = _default_scale(q.shape[-1])
    return _decode(q, k_pages, v_pages, block_table, seqlens, out, lse, scale, weights,
                   window_left, workspace, stream)


def fa_paged_evict(k_pages, v_pages, weights, block_table, seqlens, out_table, kept, new_seqlens,
                   recent: int, stream=None) -> None:
    """Enqueue the eviction: every sequence cut to budget = kept.shape[2] tokens per key head,
    its ``recent`` newest and the heaviest others, moved in order to the pages of out_table
    (int32 [B, out_pages]: free pages, or the sequence's own first ones). kept int32
    [B, Hkv, budget] gets the tokens kept (-1 behind the last), new_seqlens int32 [B] the new
    lengths."""
    import torch
    device, dtype, B, Hkv, d, page_size, num_pages, max_pages = _cache(
        k_pages, v_pages, weights, block_table, seqlens)
    if weights is None:
        raise ValueError("eviction goes by the cache's weights")
    if kept.dim() != 3 or out_table.dim() != 2:
        raise ValueError("kept must be [B, Hkv, budget] and out_table [B, out_pages]")
    budget, out_pages = _count("budget", kept.shape[2]), _count("out_pages", out_table.shape[1])
    _check("kept", kept, (B, Hkv, budget), torch.int32, device)
    _check("out_table", out_table, (B, out_pages), torch.int32, device)
    _check("new_seqlens", new_seqlens, (B,), torch.int32, device)
    _call("fa_paged_evict", _library().fa_paged_evict, device, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), weights.data_ptr(), block_table.data_ptr(),
        seqlens.data_ptr(), out_table.data_ptr(), kept.data_ptr(), new_seqlens.data_ptr(), B, Hkv,
        d, page_size, num_pages, max_pages, out_pages, budget, _count("recent", recent),
        _dtype_code(k_pages)))


def paged_evict(k_pages, v_pages, weights, block_table, seqlens, out_table, budget: int,
                recent: int, stream=None):
    """kept, new_seqlens = eviction of all but ``budget`` tokens per sequence and key head (see
    ``fa_paged_evict``); the kept tokens are then the first ones of out_table's pages."""
    import torch
    if _count("budget", budget) < 1:
        raise ValueError("budget must be at least 1")
    with _stream_of(stream, k_pages.device):
        kept = torch.empty((block_table.shape[0], k_pages.shape[2], budget), dtype=torch.int32,
                           device=k_pages.device)
        new_seqlens = torch.empty_like(seqlens)
    fa_paged_evict(k_pages, v_pages, weights, block_table, seqlens, out_table, kept, new_seqlens,
                   recent, stream)
    return kept, new_seqlens
