"""Drafted and branching sequences on the CPU: bad arguments refused on the host before any CUDA
work; the binding's own checks; rules of the sources; the plain implementations that the GPU tests
compare with, on cases worked out by hand."""
import math
import os
import re

import pytest
import torch

from draft_util import Pool, accept_ref, draft_cache, line, seen_tokens, tree_ref

NULL, SHAPE, DTYPE, ALIGN, ALIAS, SCALE, WORKSPACE = -1, -2, -3, -4, -5, -9, -11
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "io_aware_attention_fa2_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    from io_aware_attention_fa2_gb300 import binding
    from io_aware_attention_fa2_gb300 import build as fa_build
    fa_build.build()
    return binding.load_library()


# Fake, never dereferenced addresses, 1 MiB apart: every call below fails a host-side check.
A = [0x100000 * (i + 1) for i in range(16)]


def tree(lib, q=A[0], kp=A[1], vp=A[2], table=A[3], lens=A[4], parents=A[5], new=A[6], o=A[7],
         lse=A[8], B=2, T=8, Hq=4, Hkv=2, d=64, page=16, pages=8, width=400, window=-1, scale=0.1,
         dtype=0, ws=A[9], ws_bytes=1 << 62):
    return lib.fa_paged_tree(q, kp, vp, table, lens, parents, new, o, lse, B, T, Hq, Hkv, d, page,
                             pages, width, window, scale, dtype, ws, ws_bytes, None)


def accept(lib, kp=A[0], vp=A[1], weights=A[2], table=A[3], lens=A[4], parents=A[5], leaf=A[6],
           new=A[7], path=A[8], out=A[9], B=2, T=8, Hkv=2, d=64, page=16, pages=8, width=4,
           dtype=0):
    return lib.fa_paged_accept(kp, vp, weights, table, lens, parents, leaf, new, path, out, B, T,
                               Hkv, d, page, pages, width, dtype, None)


def copy(lib, kp=A[0], vp=A[1], weights=A[2], src=A[3], dst=A[4], rows=A[5], M=4, Hkv=2, d=64,
         page=16, pages=8, dtype=0):
    return lib.fa_paged_copy(kp, vp, weights, src, dst, rows, M, Hkv, d, page, pages, dtype, None)


def fork(lib, table=A[0], lens=A[1], source=A[2], refs=A[3], free=A[4], num=A[5], out=A[6],
         out_lens=A[7], src=A[8], dst=A[9], rows=A[10], B=2, C=3, page=16, pages=8, width=4):
    return lib.fa_paged_fork(table, lens, source, refs, free, num, out, out_lens, src, dst, rows,
                             B, C, page, pages, width, None)


def resize(lib, table=A[0], old=A[1], new=A[2], granted=A[3], refs=A[4], free=A[5], num=A[6], B=2,
           page=16, pages=8, width=4):
    return lib.fa_paged_resize(table, old, new, granted, refs, free, num, B, page, pages, width,
                               None)


def test_tree_workspace_sizes(lib):
    size = lib.fa_paged_tree_workspace_size
    # parts of two runs on each of 152 SMs: up to 128 rows (256 from 129 on), then the units
    assert size(16, 16, 32, 8, 128, 16, 1024) == 304 * 64 * (128 * 4 + 8) + 16 * 8 * 8
    assert size(8, 64, 32, 8, 128, 64, 512) == 304 * 256 * (128 * 4 + 8) + 8 * 8 * 8
    assert size(8, 65, 32, 8, 128, 64, 512) == 304 * 256 * (128 * 4 + 8) + 8 * 8 * 2 * 8
    assert size(1, 300, 1, 1, 64, 64, 4) == 2 * 4 * 256 * (64 * 4 + 8) + 2 * 8
    assert size(1, 300, 1, 1, 64, 64, 2) == 0                 # one tile: never split
    # clusters of 8, 4 and 2 CTAs, and one CTA, with up to four tiles of 128 tokens each
    for units, tiles in ((1, 32), (15, 32), (16, 16), (36, 16), (37, 8), (76, 8), (77, 4), (304, 4)):
        assert size(units, 8, 4, 1, 64, 128, tiles) == 0, units
        assert size(units, 8, 4, 1, 64, 128, tiles + 1) > 0, units
    assert size(305, 8, 4, 1, 64, 128, 4) > 0
    assert size(1, 129, 1, 1, 64, 128, 4) > 0                 # two row tiles
    assert size(2, 8, 8, 3, 64, 16, 10) == 0                  # 8 % 3
    assert size(2, 8, 8, 2, 64, 17, 10) == 0                  # page size
    assert size(2, 1025, 8, 2, 64, 16, 10) == 0


def test_tree_refusals(lib):
    for name in ("q", "kp", "vp", "table", "lens", "o", "lse"):
        assert tree(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(T=0), dict(T=1025), dict(Hq=0), dict(Hkv=0), dict(Hq=3),
                dict(Hq=1), dict(d=256), dict(page=48), dict(page=512), dict(pages=0),
                dict(width=0), dict(width=1 << 27), dict(B=1 << 16, T=1 << 10, Hq=32, Hkv=1),
                dict(B=1 << 11, T=1, Hq=1, Hkv=1, width=1 << 23)):
        assert tree(lib, **bad) == SHAPE, bad
    assert tree(lib, dtype=7) == DTYPE
    assert tree(lib, scale=math.nan) == SCALE
    assert tree(lib, scale=3e38) == SCALE                 # infinite in log2 units
    assert tree(lib, ws=0) == NULL
    assert tree(lib, ws_bytes=100) == WORKSPACE
    assert tree(lib, ws=A[9] + 8) == ALIGN
    assert tree(lib, ws=A[7]) == ALIAS
    assert tree(lib, o=A[7] + 2) == ALIGN
    assert tree(lib, parents=A[5] + 1) == ALIGN
    assert tree(lib, lse=A[8] + 2) == ALIGN
    assert tree(lib, o=A[0]) == ALIAS
    assert tree(lib, lse=A[5] + 4) == ALIAS
    assert tree(lib, o=A[1] + 4096) == ALIAS


def test_accept_refusals(lib):
    for name in ("kp", "vp", "table", "lens", "leaf", "path", "out"):
        assert accept(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(T=0), dict(T=1025), dict(Hkv=0), dict(d=100), dict(page=8),
                dict(pages=0), dict(width=0), dict(B=1 << 16, Hkv=1 << 15)):
        assert accept(lib, **bad) == SHAPE, bad
    assert accept(lib, dtype=2) == DTYPE
    assert accept(lib, kp=A[0] + 8) == ALIGN
    assert accept(lib, leaf=A[6] + 2) == ALIGN
    assert accept(lib, out=A[4]) == ALIAS                 # the lengths cannot be replaced in place
    assert accept(lib, path=A[5]) == ALIAS
    assert accept(lib, vp=A[0]) == ALIAS


def test_copy_refusals(lib):
    for name in ("kp", "vp", "src", "dst"):
        assert copy(lib, **{name: 0}) == NULL
    for bad in (dict(M=0), dict(Hkv=0), dict(d=32), dict(page=24), dict(pages=0),
                dict(M=1 << 30), dict(Hkv=1 << 24)):
        assert copy(lib, **bad) == SHAPE, bad
    assert copy(lib, dtype=-1) == DTYPE
    assert copy(lib, weights=A[2] + 4) == ALIGN
    assert copy(lib, rows=A[5] + 2) == ALIGN
    assert copy(lib, src=A[0] + 64) == ALIAS
    assert copy(lib, vp=A[0]) == ALIAS


def test_fork_refusals(lib):
    for name in ("table", "lens", "source", "refs", "free", "num", "out", "out_lens", "src", "dst",
                 "rows"):
        assert fork(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(C=0), dict(B=8193), dict(C=8193), dict(page=20), dict(pages=0),
                dict(width=0), dict(width=1 << 27), dict(C=8192, width=1 << 18)):
        assert fork(lib, **bad) == SHAPE, bad
    assert fork(lib, refs=A[3] + 2) == ALIGN
    assert fork(lib, out=A[0]) == ALIAS                   # the tables stay
    assert fork(lib, out_lens=A[1]) == ALIAS
    assert fork(lib, src=A[9] + 4) == ALIAS


def test_resize_refusals(lib):
    for name in ("table", "old", "new", "granted", "refs", "free", "num"):
        assert resize(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(B=8193), dict(page=20), dict(pages=0), dict(width=0),
                dict(width=1 << 27), dict(B=8192, width=1 << 18)):
        assert resize(lib, **bad) == SHAPE, bad
    assert resize(lib, num=A[6] + 1) == ALIGN
    assert resize(lib, granted=A[1]) == ALIAS
    assert resize(lib, free=A[4] + 16) == ALIAS


def test_valid_arguments_without_gpu_fail_in_device_query(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; the GPU tests cover real launches")
    for call in (tree, accept, copy, fork, resize):
        assert call(lib) in (-6, -10), call


def test_binding_refuses_what_is_not_a_cuda_tensor():
    import io_aware_attention_fa2_gb300 as fa
    c = draft_cache([5], [3], 16, 2, 64, "bf16", device="cpu")
    q = torch.zeros((1, 3, 4, 64), dtype=torch.bfloat16)
    parents = torch.full((1, 3), -1, dtype=torch.int32)
    pool = fa.new_page_pool(8, device="cpu")
    assert pool.free_pages.tolist() == [7, 6, 5, 4, 3, 2, 1, 0] and pool.num_free.tolist() == [8]
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_tree_attention(q, c.k, c.v, c.table, c.seqlens, parents=parents)
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_accept(c.k, c.v, c.table, c.seqlens, one, parents)
    with pytest.raises(ValueError, match="k_pages"):
        fa.fa_paged_copy(c.k, c.v, one, one)
    with pytest.raises(ValueError, match="block_table"):
        fa.paged_fork(pool, c.table, c.seqlens, one, 16)
    with pytest.raises(ValueError, match="block_table"):
        fa.paged_resize(pool, c.table, c.seqlens, one, 16)
    with pytest.raises(ValueError, match="num_pages"):
        fa.new_page_pool(0, device="cpu")


# ------------------------------------------------------------------------------------- sources
def sources():
    """File name -> text without comments, of the files that launch the cache's kernels."""
    out = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = open(os.path.join(CSRC, name)).read()
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
            if "launch_paged(" in text and name != "fa_paged.cuh":
                out[name] = text
    return out


def test_chained_kernels_of_drafts_and_forks():
    """Every kernel waits for the one before it, which may still write its inputs: none of them is
    declared read-only or read through the non-coherent path; launches report their own status."""
    assert {"fa_paged_tree.cu", "fa_paged_pool.cu"} <= set(sources())
    for name, text in sources().items():
        for word in ("__restrict__", "__ldg", ".nc", "restrict", "<<<", "cudaGetLastError"):
            assert word not in text, (name, word)
        assert not re.search(r"__ld(cg|ca|cs|cv|lu)\b", text), name
        assert text.count("__global__") == text.count("  wait_prerequisites();"), name


# ------------------------------------------------------------------------- plain forms by hand
def test_line_and_seen_tokens_by_hand():
    parents = [-1, 0, 0, 2, -1, 3]
    assert line(parents, 5) == [0, 2, 3, 5] and line(parents, 4) == [4]
    assert line(None, 2) == [0, 1, 2]
    assert line([-1, 1, 7], 2) == [2] and line([-1, 1], 1) == [1]   # no earlier tokens
    assert seen_tokens(2, parents, 5, -1) == [0, 1, 2, 4, 5, 7]
    # token 5 stands at position 5, its ancestors at 2, 3 and 4
    assert seen_tokens(2, parents, 5, 2) == [4, 5, 7]
    assert seen_tokens(2, parents, 5, 4) == [1, 2, 4, 5, 7]
    assert seen_tokens(0, parents, 4, 0) == [4]


def test_plain_tree_by_hand():
    """A context token and two drafted siblings, scores 0, ln 3, ln 3: each sees two tokens."""
    c = draft_cache([1], [2], 16, 1, 64, "bf16", device="cpu")
    c.k[:], c.v[:] = 0, 0
    pg = int(c.table[0, 0])
    c.k[pg, 1:3, 0, 0] = 1.0
    c.v[pg, :3, 0, 5] = torch.tensor([8.0, 16.0, 40.0])
    q = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    o, lse, *_ = tree_ref(c, q, math.log(3.0), torch.tensor([[-1, -1]]))
    assert torch.allclose(o[0, :, 0, 5], torch.tensor([14.0, 32.0], dtype=torch.float64))
    assert torch.allclose(lse[0, 0], torch.full((2,), math.log(4.0), dtype=torch.float64))


def test_plain_accept_by_hand():
    c = draft_cache([15], [4], 16, 1, 64, "bf16", weights=True, device="cpu")
    first, second = (int(x) for x in c.table[0, :2])
    path, lens, k, _, w = accept_ref(c, torch.tensor([[-1, -1, 1, 1]]), [3], 4)
    assert path.tolist() == [[1, 3, -1, -1]] and lens.tolist() == [17]
    assert torch.equal(k[first, 15], c.k[second, 0]) and torch.equal(k[second, 0], c.k[second, 2])
    assert float(w[first, 0, 15]) == float(c.w[second, 0, 0])


def test_plain_pool_by_hand():
    pool = Pool(6)
    table = [[-1] * 3, [-1] * 3]
    assert pool.resize(table, [0, 0], [20, 16], 16) == [20, 16]
    assert table == [[0, 1, -1], [2, -1, -1]] and pool.free == [5, 4, 3]
    out = pool.fork(table, [20, 16], [0, 1, 0, -1], 16)
    assert out[0] == [[0, 3, -1], [2, -1, -1], [0, 4, -1], [-1] * 3]
    assert out[1:] == ([20, 16, 20, 0], [1, -1, 1, -1], [3, -1, 4, -1], [4, 0, 4, 0])
    assert pool.refs == [3, 1, 2, 1, 1, 0] and pool.free == [5]
    assert pool.fork(table, [20, 16], [0, 0], 16)[1] == [20, -1]
    assert pool.resize(table, [20, 16], [0, 48], 16) == [0, 16]   # page 0 has other holders
    assert table == [[-1] * 3, [2, -1, -1]] and pool.free == [1]
