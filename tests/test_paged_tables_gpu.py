"""Block tables as a serving program keeps them: pages that were given back in front of a window,
prefixes shared between sequences, destinations among the sequence's own pages."""
import pytest
import torch

from paged_util import Cache, check_decode, decode_ref, default_scale, evict_ref, same_bits
from test_paged_gpu import check_evict, check_weights, free_table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


@pytest.mark.parametrize("n,window", [(200, 30), (5000, 1000), (5000, 0), (9001, 4095)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_pages_in_front_of_a_window_are_given_back(n, window, page):
    """Their entries name no page, or one of another sequence: they are not followed, and no
    error is recorded."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([n, n - 7], page, 2, 64, "bf16", seed=n, weights=True)
    for b in range(2):
        first = max(0, c.lens[b] - 1 - window) // page
        c.table[b, :first] = -1 if b == 0 else 2 ** 31 - 1
    q = c.query(8)
    before = c.w.clone()
    o, lse = fa.paged_attention(q, c.k, c.v, c.table, c.seqlens, weights=c.w, window_left=window)
    ref = decode_ref(c, q, default_scale(64), window)
    check_decode(c, q, o, lse, ref, (n, window, page))
    check_weights(c, before, ref)


@pytest.mark.parametrize("d", [64, 128])
def test_evict_sequences_that_share_a_prefix(d):
    """Into free pages: the shared pages are read by both and stay as they are."""
    c = Cache([700, 500, 333], 32, 2, d, "fp16", seed=d, weights=True, spare=24)
    c.table[1, :6] = c.table[0, :6]
    c.table[2, :10] = c.table[0, :10]
    check_evict(c, free_table(c, 250), 250, 60)


@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("d,page", [(64, 64), (128, 256)])
def test_evict_into_earlier_own_pages_in_several_rounds(d, page, shift):
    """Destinations shifted back among the sequence's own pages, more tokens than a round of the
    move takes: a row may be written only after the rounds that read it."""
    n, budget = 24000, 20000
    c = Cache([n], page, 2, d, "bf16", seed=d + shift, weights=True, spare=shift)
    used = -(-budget // page)
    out = torch.cat([c.free[:shift].cuda(), c.table[0, :used - shift]]).view(1, used).contiguous()
    check_evict(c, out, budget, 100)


def test_evict_of_short_sequences_into_earlier_own_pages():
    """Nothing to select: every row moves by a page, in several rounds."""
    c = Cache([9000], 64, 1, 64, "fp16", seed=2, weights=True, spare=1)
    out = torch.cat([c.free[:1].cuda(), c.table[0, :-1]]).view(1, -1).contiguous()
    assert out.shape[1] * 64 >= 9000
    check_evict(c, out, 9000, 0)


def test_evict_with_pages_behind_the_length_as_destinations():
    """Pages of the table that hold no token yet are as good as free ones."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([300], 16, 2, 64, "bf16", seed=5, weights=True, spare=10, max_pages=40)
    c.table[0, 19:29] = c.free[:10].cuda()
    out = c.table[:, 19:29].contiguous()
    kept, lens, k, v, w = evict_ref(c, out, 150, 20)
    got = fa.paged_evict(c.k, c.v, c.w, c.table, c.seqlens, out, 150, 20)
    assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), lens)
    assert same_bits(c.k, k) and same_bits(c.v, v) and same_bits(c.w, w)
