"""Shapes whose products pass 64 bits are refused on the host like any other that is too large: a
product that has wrapped around may look like a small one."""
import pytest

from test_draft import A, SHAPE, lib, tree   # noqa: F401  (lib: a fixture)
from test_paged import decode

BIG = 1 << 30


@pytest.mark.parametrize("shape", [
    dict(B=BIG, T=1024, Hq=BIG, Hkv=1, width=16),            # rows 2^70, tiles 9 * 2^64
    dict(B=BIG, T=1024, Hq=BIG, Hkv=1 << 20, width=16),      # tiles 9 * 2^74
    dict(B=1 << 27, T=1024, Hq=1 << 27, Hkv=1, width=16),    # rows 2^64
    dict(B=BIG, T=64, Hq=1 << 28, Hkv=1 << 20, width=1 << 26),
    dict(B=(1 << 31) - 1, T=1024, Hq=(1 << 31) - 1, Hkv=1, width=1)])
def test_tree(lib, shape):   # noqa: F811
    assert tree(lib, **shape) == SHAPE
    assert lib.fa_paged_tree_workspace_size(shape["B"], shape["T"], shape["Hq"], shape["Hkv"], 64, 16,
                                            shape["width"]) == 0


@pytest.mark.parametrize("shape", [
    dict(B=BIG, Hq=BIG, Hkv=1, width=14 * 64),               # 2^60 * (14 + 2)
    dict(B=1 << 24, Hq=BIG, Hkv=1 << 6, width=(1 << 16) - 128),   # 2^54 * 2^10
    dict(B=1 << 23, Hq=1 << 23, Hkv=1, width=(1 << 24) - 128)])   # 2^46 * 2^18
def test_decode(lib, shape):   # noqa: F811
    assert decode(lib, **shape) == SHAPE
    assert lib.fa_paged_decode_workspace_size(shape["B"], shape["Hq"], shape["Hkv"], 64, 16,
                                              shape["width"], 1) == 0


def test_largest_shapes_that_pass(lib):   # noqa: F811
    """These get as far as the spans or the device."""
    assert tree(lib, B=1 << 20, T=1, Hq=2, Hkv=1, width=1) != SHAPE
    assert tree(lib, B=1, T=1024, Hq=(1 << 21) - 1, Hkv=(1 << 21) - 1, width=1, d=64) == SHAPE  # a page
    assert tree(lib, B=1, T=1024, Hq=1 << 20, Hkv=1 << 10, width=1) != SHAPE
    assert tree(lib, B=1, T=1024, Hq=1 << 21, Hkv=1 << 10, width=1) == SHAPE         # 2^31 rows
    assert decode(lib, B=1 << 20, Hq=1 << 9, Hkv=1, width=64) != SHAPE
    assert decode(lib, B=1 << 20, Hq=1 << 10, Hkv=1, width=64) == SHAPE
