"""Decoding over the paged cache at the edges of its numbers: infinite values, probabilities far
below the largest one, arguments at the ends of their ranges."""
import math

import pytest
import torch

from paged_util import Cache, check_decode, decode_ref, default_scale, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens", [[1], [40, 7], [3000, 1, 900]])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
def test_infinite_values(d, dtype, lens, weights):
    """A visible infinite value makes its column of O infinite, of its sign; two of both signs,
    or a NaN, make it NaN; the other columns, LSE and the weights are as ever. Where the window
    hides the token the value does not matter."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache(lens, 16, 2, d, dtype, seed=len(lens) + d, weights=weights)
    q = c.query(8)
    plain = c.v.clone()
    for b, n in enumerate(lens):
        pg, row = c.rows(c.table, b, n)
        for t, col, value in ((0, 3, math.inf), (n // 2, 5, -math.inf), (n - 1, 7, math.inf),
                              (0, d - 1, math.nan), (n // 3, 9, math.inf), (n - 1, 9, -math.inf)):
            c.v[pg[t], row[t], :, col] = value
    o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens,
                                weights=None if c.w is None else c.w.clone())
    ref = decode_ref(c, q, default_scale(d))
    want, bound = ref[0], ref[3]
    finite = torch.isfinite(want)
    assert not finite[:, :, [3, 5, 7, d - 1]].any() and torch.isneginf(want[..., 5]).all()
    got = o.double().cpu()
    assert ((got - want).abs()[finite] <= bound[finite]).all()
    assert torch.equal(got[~finite].nan_to_num(nan=7.0), want[~finite].nan_to_num(nan=7.0))
    assert ((lse.double().cpu() - ref[1]).abs() <= ref[4]).all()
    # one visible token, whose values are finite in these columns
    o0, _ = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, window_left=0)
    for b, n in enumerate(lens):
        pg, row = c.rows(c.table, b, n)
        last = plain[pg[-1], row[-1]].repeat_interleave(4, 0)
        cols = [x for x in range(d) if n > 1 and x not in (7, 9)]
        assert same_bits(o0[b][:, cols].contiguous(), last[:, cols].contiguous())


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "fp16"), (64, "bf16")])
def test_many_small_probabilities_behind_heavy_tokens(d, dtype):
    """Four heavy tokens with small values in front, all others e^-18 (below fp16's 2^-25) as
    probable: what these add up to is most of O. 320 units, so that a run is a whole sequence and
    every warp of it meets a heavy token in the first tile."""
    import io_aware_attention_fa2_gb300 as fa
    B, Hkv, n = 40, 8, 1024
    c = Cache([n] * B, 256, Hkv, d, dtype, seed=d)
    for b in range(B):
        pg, row = c.rows(c.table, b, n)
        c.k[pg, row] = 0
        c.v[pg, row] *= 100
        c.v[pg, row] += 1000
        heavy = torch.arange(0, 64, 16)
        c.k[pg[heavy], row[heavy], :, 0] = 18.0
        c.v[pg[heavy], row[heavy]] *= 2.0 ** -20
    q = c.query(Hkv) * 0
    q[..., 0] = 1.0
    o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, scale=1.0)
    check_decode(c, q, o, lse, decode_ref(c, q, 1.0), (d, dtype))


@pytest.mark.parametrize("d", [64, 128])
def test_largest_fp16_numbers(d):
    """Values at the type's largest number, all probabilities equal: sums far past fp16."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([5000, 130, 1], 64, 1, d, "fp16", seed=3, weights=True)
    for b, n in enumerate(c.lens):
        pg, row = c.rows(c.table, b, n)
        c.v[pg, row] = torch.finfo(torch.float16).max
    q = c.query(4) * 0
    o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, weights=c.w)
    assert (o == torch.finfo(torch.float16).max).all()
    want = torch.log(c.seqlens.double())[:, None].expand(3, 4)
    assert ((lse.double() - want).abs() <= 2.0 ** -20 + want * 2.0 ** -22).all()


def test_integers_past_32_bits():
    """A window past every length is none; counts that the library's ints cannot hold are
    refused, not cut to their low 32 bits."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([300], 16, 1, 64, "bf16", seed=4, weights=True, spare=20)
    q = c.query(2)
    want = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens)
    for window in (2 ** 32, 2 ** 31, 2 ** 63 - 1, 2 ** 31 - 1, -1, -2 ** 31, -2 ** 32 + 5):
        o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, window_left=window)
        assert same_bits(o, want[0]) and same_bits(lse, want[1]), window
    p = torch.randn((1, 200, 1, 64), generator=c.g).to(c.dtype).cuda()
    lse = torch.full((1, 1, 200), 6.0, device="cuda")
    w = fa.key_weights(p, p, lse)
    for window in ((2 ** 32, 2 ** 33), (2 ** 31, -1), (-2 ** 32, -2 ** 40 + 3)):
        assert same_bits(fa.key_weights(p, p, lse, window=window), w), window
    out = c.free[:4].view(1, 4).cuda()
    before = [x.clone() for x in (c.k, c.v, c.w)]
    for budget, recent in ((50, 2 ** 32 + 5), (50, -2 ** 32 + 5), (2 ** 32 + 5, 2)):
        with pytest.raises(ValueError, match="out of range"):
            fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, out, budget, recent)
    with pytest.raises(ValueError, match="too large"):
        wide = torch.empty((1, 2 ** 32 + 19), dtype=torch.int32, device="cuda")
        fa.paged_attention(q, c.k, c.v, wide, c.seqlens)
    del wide
    torch.cuda.empty_cache()
    for x, y in zip((c.k, c.v, c.w), before):
        assert same_bits(x, y)


@pytest.mark.parametrize("side", [False, True])
def test_key_weights_take_the_lengths_that_the_forward_takes(side):
    """Host lengths and other integer types, as attention_forward accepts them."""
    import io_aware_attention_fa2_gb300 as fa
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((2, 300, 2, 64), generator=g).to(torch.bfloat16).cuda()
               for _ in range(3))
    lens = torch.tensor([300, 77])
    _, lse = fa.attention_forward(q, k, v, causal=True, seqlens_k=lens)
    want = fa.key_weights(q, k, lse, causal=True, seqlens_k=lens.to(torch.int32).cuda())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    for given in (lens, lens.to(torch.int32), lens.cuda()):
        torch.cuda.synchronize()
        got = fa.key_weights(q, k, lse, causal=True, seqlens_k=given, stream=stream)
        torch.cuda.synchronize()
        assert same_bits(got, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens", [[100], [3000, 64]])
def test_large_scores(dtype, lens):
    """Equal scores from 2^9 to 2^31 (log2 units), where a step of fp32 is up to 256: the
    probabilities are equal all the same, and O is the mean of the values."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache(lens, 16, 1, 64, dtype, seed=11, weights=True)
    q = c.query(3) * 0
    q[..., 0] = 2.0 ** 15
    for b, n in enumerate(lens):
        pg, row = c.rows(c.table, b, n)
        c.k[pg, row] = 0
        c.k[pg, row, :, 0] = 2.0 ** 15
    half = torch.finfo(c.dtype).eps / 2
    for e in range(-21, 1):
        for sign in (1.0, -1.0):
            w = c.w.clone()
            o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, scale=sign * 0.7 * 2.0 ** e,
                                        weights=w)
            for b, n in enumerate(lens):
                pg, row = c.rows(c.table, b, n)
                v = c.v[pg, row, 0].double()
                want, size = v.mean(0), v.abs().mean(0)
                # the output's rounding; P in two parts and sums in 32 bits
                bound = half * want.abs() + 2.0 ** -15 * size
                assert ((o[b].double() - want).abs() <= bound).all(), (e, sign)
                s = sign * 0.7 * 2.0 ** (e + 30)
                assert ((lse[b].double() - s - math.log(n)).abs() <= abs(s) * 2.0 ** -22
                        + 2.0 ** -19).all(), (e, sign)
                added = (w[pg, :, row] - c.w[pg, :, row]).double()
                assert (added - 3.0 / n).abs().max() <= 2.0 ** -18 / n + 2.0 ** -23, (e, sign)
