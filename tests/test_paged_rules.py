"""The rules that choose a path of the paged cache's operators, as their workspace sizes show
them, on the CPU."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from io_aware_attention_fa2_gb300 import binding
    from io_aware_attention_fa2_gb300 import build as fa_build
    fa_build.build()
    return binding.load_library()


@pytest.mark.parametrize("d,tiles,units", [
    (128, 32, 15), (128, 17, 15), (128, 16, 36), (128, 9, 36), (128, 8, 76), (128, 5, 76),
    (128, 4, 304), (128, 1, 304), (64, 32, 36), (64, 16, 74), (64, 8, 152), (64, 4, 608)])
def test_short_calls_take_as_many_units_as_run_at_once(lib, d, tiles, units):
    """A unit in a cluster of eight, four, two or (in two turns) one CTA of four tiles each, as
    long as all clusters run at once: 8 x 15 CTAs at d = 128, not 152, since a cluster cannot
    span the groups of SMs. One unit more, or one tile more than the clusters hold, takes runs,
    which need a workspace."""
    def need(units, tiles):
        return lib.fa_paged_decode_workspace_size(units, 1, 1, d, 64, tiles, 0)
    assert need(units, tiles) == 0
    assert need(units + 1, tiles) > 0
    if tiles in (32, 16, 8, 4):
        assert need(units, tiles + 1) > 0


def test_key_weights_index_sums_stay_within_int(lib):
    """The largest key index that a CTA forms, N rounded up to 256, less one, plus a window as wide
    as the sequence, plus one: within 32 bits for every length that is accepted."""
    def call(N):   # one byte of workspace: an accepted length stops there
        a = [0x100000 * (i + 1) for i in range(5)]
        return lib.fa_key_weights(*a[:4], 1, 2, 1, N, 64, 1, 2 ** 31 - 1, -1, None, 0.1, 0, a[4], 1,
                                  None)
    most = max(N for N in range((1 << 30) - 300, (1 << 30) + 300) if call(N) == -11)
    assert call(most + 1) == -2
    assert -(-most // 256) * 256 - 1 + most + 1 < 2 ** 31


def test_messages_name_what_the_call_needs(lib):
    from io_aware_attention_fa2_gb300 import FaError
    for where, size in (("fa_paged_decode", "fa_paged_decode_workspace_size"),
                        ("fa_key_weights", "fa_key_weights_workspace_size"),
                        ("fa_bwd_masked", "fa_bwd_workspace_size"),
                        ("fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size")):
        e = FaError(-11, where)
        assert e.code == -11
        assert str(e) == "%s failed: workspace smaller than %s() (-11)" % (where, size)
        assert hasattr(lib, size)
    assert "pages of 16, 32, 64, 128 or 256" in str(FaError(-2, "fa_paged_decode"))
