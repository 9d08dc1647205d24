"""Fork of a sequence whose last page, filled in part, is no page of the pool: passed on as -1 and
recorded by the fork itself, without a page or a copy for it; so is a stack's entry that is no page."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FA_ERR_PAGE = -13


@pytest.fixture(autouse=True)
def no_error_left():
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    yield
    assert fa.device_error() == 0


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("width", [4, 3000])          # one launch, and two
@pytest.mark.parametrize("entry", [-1, -9, 12, 10 ** 9])
def test_a_last_page_outside_the_pool(width, entry):
    import io_aware_attention_fa2_gb300 as fa
    pool = fa.PagePool(int32([1, 1, 1, 1] + [0] * 8), int32([11, 10, 9, 8, 7, 6, 5, 4] + [-1] * 4),
                       int32([8]))
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, :3], table[1, :2] = int32([0, 1, entry]), int32([2, 3])
    out = fa.paged_fork(pool, table, int32([40, 20]), int32([1, 0, 0, 1]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert out.seqlens.tolist() == [20, 40, 40, 20]
    assert out.block_table[:, :3].tolist() == [[2, 4, -1], [0, 1, -1], [0, 1, -1], [2, 5, -1]]
    assert (out.block_table[:, 3:] == -1).all()
    assert out.copy_src.tolist() == [3, -1, -1, 3]
    assert out.copy_dst.tolist() == [4, -1, -1, 5]
    assert out.copy_rows.tolist() == [4, 0, 0, 4]
    assert pool.num_free.tolist() == [6]
    assert pool.refs.tolist() == [3, 3, 3, 1, 1, 1] + [0] * 6
    assert pool.free_pages.tolist() == [11, 10, 9, 8, 7, 6] + [-1] * 6
    k = torch.zeros((12, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    fa.fa_paged_copy(k, k.clone(), out.copy_src, out.copy_dst, rows=out.copy_rows)
    assert fa.device_error() == 0                      # the list of copies is a good one


@pytest.mark.parametrize("entry", [-3, 12])
def test_a_stack_with_a_bad_entry(entry):
    """The sequence that gets it has no last page and no copy."""
    import io_aware_attention_fa2_gb300 as fa
    pool = fa.PagePool(int32([1] + [0] * 11), int32([5, 4, 3, entry, 2] + [-1] * 7), int32([5]))
    out = fa.paged_fork(pool, int32([[0, -1]]), int32([5]), int32([0, 0, 0]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert out.seqlens.tolist() == [5, 5, 5]
    assert out.block_table.tolist() == [[2, -1], [-1, -1], [3, -1]]
    assert out.copy_src.tolist() == [0, -1, 0]
    assert out.copy_dst.tolist() == [2, -1, 3]
    assert out.copy_rows.tolist() == [5, 0, 5]
    assert pool.num_free.tolist() == [2] and pool.free_pages.tolist() == [5, 4] + [-1] * 10


def test_an_empty_pool_and_a_bad_last_page():
    """It needs no page from the pool, so it is passed on where a good one gets nothing."""
    import io_aware_attention_fa2_gb300 as fa
    pool = fa.PagePool(int32([1, 1]), int32([-1, -1]), int32([0]))
    out = fa.paged_fork(pool, int32([[0, 7], [1, -1]]), int32([20, 5]), int32([0, 1]), 16)
    assert fa.device_error() == FA_ERR_PAGE
    assert out.seqlens.tolist() == [20, -1]
    assert out.block_table.tolist() == [[0, -1], [-1, -1]]
    assert out.copy_dst.tolist() == [-1, -1] and pool.refs.tolist() == [2, 1]
