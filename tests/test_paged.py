"""The paged cache's entry points on the CPU: workspace sizes, and bad arguments refused on the
host before any CUDA work; the binding's own checks; the plain implementations the GPU tests
compare with, on cases worked out by hand."""
import math

import pytest
import torch

from paged_util import Cache, decode_ref, evict_ref, key_weights_ref

NULL, SHAPE, DTYPE, ALIGN, ALIAS, SCALE, WORKSPACE = -1, -2, -3, -4, -5, -9, -11
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from io_aware_attention_fa2_gb300 import binding
    from io_aware_attention_fa2_gb300 import build as fa_build
    fa_build.build()
    return binding.load_library()


# Fake, never dereferenced addresses, 1 MiB apart: every call below fails a host-side check.
A = [0x100000 * (i + 1) for i in range(16)]


def key_weights(lib, q=A[0], k=A[1], lse=A[2], w=A[3], B=1, Hq=4, Hkv=2, N=100, d=64, causal=1,
                left=-1, right=-1, lens=None, scale=0.1, dtype=0, ws=A[4], ws_bytes=1 << 16):
    return lib.fa_key_weights(q, k, lse, w, B, Hq, Hkv, N, d, causal, left, right, lens, scale,
                              dtype, ws, ws_bytes, None)


def append(lib, k=A[0], v=A[1], w=A[2], kp=A[3], vp=A[4], weights=A[5], table=A[6], lens=A[7],
           new=A[8], B=2, N=3, Hkv=2, d=64, page=16, pages=8, width=4, dtype=0):
    return lib.fa_paged_append(k, v, w, kp, vp, weights, table, lens, new, B, N, Hkv, d, page,
                               pages, width, dtype, None)


def decode(lib, q=A[0], kp=A[1], vp=A[2], weights=A[3], table=A[4], lens=A[5], o=A[6], lse=A[7],
           B=2, Hq=4, Hkv=2, d=64, page=16, pages=8, width=400, window=-1, scale=0.1, dtype=0,
           ws=A[8], ws_bytes=1 << 62):
    return lib.fa_paged_decode(q, kp, vp, weights, table, lens, o, lse, B, Hq, Hkv, d, page,
                               pages, width, window, scale, dtype, ws, ws_bytes, None)


def evict(lib, kp=A[0], vp=A[1], weights=A[2], table=A[3], lens=A[4], out=A[5], kept=A[6],
          new=A[7], B=2, Hkv=2, d=64, page=16, pages=8, width=4, out_pages=2, budget=20, recent=5,
          dtype=0):
    return lib.fa_paged_evict(kp, vp, weights, table, lens, out, kept, new, B, Hkv, d, page, pages,
                              width, out_pages, budget, recent, dtype, None)


def test_workspace_sizes(lib):
    assert lib.fa_key_weights_workspace_size(2, 8, 2, 100) == 2 * 8 * 100 * 4
    assert lib.fa_key_weights_workspace_size(2, 8, 8, 100) == 0
    assert lib.fa_key_weights_workspace_size(0, 8, 2, 100) == 0
    small = lib.fa_paged_decode_workspace_size(2, 8, 2, 64, 16, 200, 0)
    with_w = lib.fa_paged_decode_workspace_size(2, 8, 2, 64, 16, 200, 1)
    # 50 tiles for each of 4 units: 200 runs of 4 heads' parts, then the scores
    assert small == 2 * 200 * 4 * (64 * 4 + 8) + 4 * 8
    assert with_w == small + 16 * 8 + 16 * 3200 * 4
    assert lib.fa_paged_decode_workspace_size(2, 8, 2, 64, 16, 128, 1) == 0   # 32 tiles: short
    assert lib.fa_paged_decode_workspace_size(2, 8, 2, 64, 16, 129, 1) > 0
    assert lib.fa_paged_decode_workspace_size(40, 8, 2, 64, 16, 32, 0) == 0   # 80 units, two CTAs
    assert lib.fa_paged_decode_workspace_size(40, 8, 2, 64, 16, 33, 0) > 0
    assert lib.fa_paged_decode_workspace_size(40, 8, 2, 128, 16, 16, 0) == 0  # one CTA
    assert lib.fa_paged_decode_workspace_size(40, 8, 2, 128, 16, 17, 0) > 0
    for d, units in ((64, 608), (128, 304)):                                  # two turns of one CTA
        assert lib.fa_paged_decode_workspace_size(units, 4, 1, d, 16, 16, 1) == 0
        assert lib.fa_paged_decode_workspace_size(units, 4, 1, d, 16, 17, 1) > 0
        assert lib.fa_paged_decode_workspace_size(units + 1, 4, 1, d, 16, 16, 1) > 0
    assert lib.fa_paged_decode_workspace_size(1, 32, 1, 64, 16, 16, 0) == 0   # two blocks of heads
    assert lib.fa_paged_decode_workspace_size(1, 32, 1, 64, 16, 16, 1) > 0
    assert lib.fa_paged_decode_workspace_size(2, 8, 3, 64, 16, 10, 0) == 0    # 8 % 3
    assert lib.fa_paged_decode_workspace_size(2, 8, 2, 64, 17, 10, 0) == 0    # page size
    assert lib.fa_error_string(-13) == \
        b"a block table or length named a token outside the paged cache"


def test_key_weights_refusals(lib):
    for name in ("q", "k", "lse", "w"):
        assert key_weights(lib, **{name: 0}) == NULL
    assert key_weights(lib, ws=0) == NULL
    assert key_weights(lib, ws_bytes=1599) == WORKSPACE
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(N=0), dict(d=96), dict(Hq=3),
                dict(Hq=1, Hkv=2), dict(B=1 << 16, Hq=1 << 15, Hkv=1), dict(N=(1 << 30) + 1),
                dict(N=-5)):
        assert key_weights(lib, **bad) == SHAPE, bad
    assert key_weights(lib, dtype=2) == DTYPE
    assert key_weights(lib, scale=NAN) == SCALE
    assert key_weights(lib, scale=3e38) == SCALE          # infinite in log2 units
    assert key_weights(lib, q=A[0] + 8) == ALIGN
    assert key_weights(lib, ws=A[4] + 4) == ALIGN
    assert key_weights(lib, lens=A[5] + 2) == ALIGN
    assert key_weights(lib, w=A[2] + 64) == ALIAS
    assert key_weights(lib, ws=A[3]) == ALIAS
    assert key_weights(lib, lens=A[3] + 4) == ALIAS


def test_append_refusals(lib):
    for name in ("k", "v", "kp", "vp", "table", "lens"):
        assert append(lib, **{name: 0}) == NULL
    assert append(lib, weights=0) == NULL                 # w without weights
    for bad in (dict(B=0), dict(N=0), dict(Hkv=0), dict(d=32), dict(page=8), dict(page=24),
                dict(page=512), dict(pages=0), dict(width=0), dict(width=1 << 27),
                dict(B=1 << 16, N=1 << 15), dict(Hkv=1 << 24)):
        assert append(lib, **bad) == SHAPE, bad
    assert append(lib, dtype=-1) == DTYPE
    assert append(lib, kp=A[3] + 8) == ALIGN
    assert append(lib, table=A[6] + 1) == ALIGN
    assert append(lib, vp=A[3] + 32768 - 16) == ALIAS     # pools of 8 * 16 * 2 * 64 * 2 bytes
    assert append(lib, k=A[3]) == ALIAS
    assert append(lib, lens=A[5]) == ALIAS                # lengths inside weights


def test_decode_refusals(lib):
    for name in ("q", "kp", "vp", "table", "lens", "o", "lse", "ws"):
        assert decode(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(Hq=1), dict(d=256),
                dict(page=48), dict(pages=-1), dict(width=0), dict(B=1 << 16, Hq=1 << 15, Hkv=1),
                dict(B=1 << 14, Hq=1 << 10, Hkv=1, width=1 << 13)):
        assert decode(lib, **bad) == SHAPE, bad
    assert decode(lib, dtype=7) == DTYPE
    assert decode(lib, scale=math.inf) == SCALE
    assert decode(lib, ws_bytes=0) == WORKSPACE
    assert decode(lib, o=A[6] + 2) == ALIGN
    assert decode(lib, ws=A[8] + 8) == ALIGN
    assert decode(lib, lse=A[7] + 2) == ALIGN
    assert decode(lib, o=A[0]) == ALIAS
    assert decode(lib, weights=A[1] + 4096) == ALIAS
    assert decode(lib, ws=A[6]) == ALIAS
    assert decode(lib, lse=A[5] + 4) == ALIAS


def test_evict_refusals(lib):
    for name in ("kp", "vp", "weights", "table", "lens", "out", "kept", "new"):
        assert evict(lib, **{name: 0}) == NULL
    for bad in (dict(B=0), dict(Hkv=0), dict(d=100), dict(page=0), dict(pages=0), dict(width=0),
                dict(out_pages=0), dict(budget=0), dict(budget=33), dict(recent=-1),
                dict(recent=21), dict(out_pages=1 << 27), dict(B=1 << 14, Hkv=1 << 14)):
        assert evict(lib, **bad) == SHAPE, bad
    assert evict(lib, dtype=3) == DTYPE
    assert evict(lib, vp=A[1] + 4) == ALIGN
    assert evict(lib, kept=A[6] + 2) == ALIGN
    assert evict(lib, new=A[4]) == ALIAS                  # the lengths cannot be replaced in place
    assert evict(lib, kept=A[5]) == ALIAS
    assert evict(lib, vp=A[0]) == ALIAS


def test_valid_arguments_without_gpu_fail_in_device_query(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; the GPU tests cover real launches")
    for call in (key_weights, append, decode, evict):
        assert call(lib) in (-6, -10), call


def test_binding_refuses_what_is_not_a_cuda_tensor():
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([5], 16, 2, 64, "bf16", weights=True, device="cpu")
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_attention(c.query(4), c.k, c.v, c.table, c.seqlens)
    with pytest.raises(ValueError, match="k_pages"):
        fa.fa_paged_append(c.k, c.v, c.k, c.v, c.table, c.seqlens)
    with pytest.raises(ValueError, match="budget"):
        fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, c.table, 0, 0)
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, c.table, 4, 0)
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must"):
        fa.key_weights(q, q, torch.zeros((1, 2, 4)))


def test_plain_decode_by_hand():
    """Two tokens with scores 0 and ln 3: probabilities 1/4 and 3/4."""
    c = Cache([2], 16, 1, 64, "bf16", device="cpu")
    c.k[:], c.v[:] = 0, 0
    pg = int(c.table[0, 0])
    c.k[pg, 1, 0, 0] = 1.0
    c.v[pg, 0, 0, 5], c.v[pg, 1, 0, 5] = 8.0, 16.0
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    q[0, 0, 0] = 1.0
    o, lse, added, *_ = decode_ref(c, q, math.log(3.0))
    assert abs(float(o[0, 0, 5]) - 14.0) < 1e-12 and abs(float(lse) - math.log(4.0)) < 1e-12
    assert torch.allclose(added[0], torch.tensor([[0.25, 0.75]], dtype=torch.float64))


def test_plain_key_weights_by_hand():
    """Uniform scores, causal: query i gives 1 / (i + 1) to each of its keys."""
    q = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16)
    lse = torch.log(torch.tensor([1.0, 2.0, 3.0])).expand(1, 2, 3)
    w, _ = key_weights_ref(q, q[:, :, :1], lse, 1.0, causal=True)
    want = 2 * torch.tensor([1 + 1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3], dtype=torch.float64)
    assert torch.allclose(w[0, 0], want, atol=1e-6)


def test_plain_evict_by_hand():
    c = Cache([6], 16, 1, 64, "bf16", weights=True, device="cpu")
    pg = int(c.table[0, 0])
    c.w[pg, 0, :6] = torch.tensor([0.5, NAN, 2.0, 0.5, -math.inf, 0.0])
    kept, lens, k, _, w = evict_ref(c, c.table, 3, 1)
    assert kept.tolist() == [[[0, 2, 5]]] and lens.tolist() == [3]
    assert torch.equal(k[pg, 1], c.k[pg, 2]) and w[pg, 0, :3].tolist() == [0.5, 2.0, 0.0]
