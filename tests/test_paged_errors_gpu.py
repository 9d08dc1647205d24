"""The device error word while calls on other streams record errors in it."""
import threading
import time

import pytest
import torch

from paged_util import Cache

pytestmark = pytest.mark.gpu
FA_ERR_PAGE = -13


@pytest.mark.parametrize("op", ["append", "decode"])
def test_no_error_is_lost_to_a_query_at_the_same_time(op):
    """One thread asks for errors all the time, another makes bad calls on a stream of its own:
    every one of them is reported to one of the queries that end after it."""
    import io_aware_attention_fa2_gb300 as fa
    c = Cache([40], 16, 1, 64, "bf16", seed=1)
    c.table[0, 1] = c.num_pages
    q = c.query(1)
    k = torch.zeros((1, 30, 1, 64), dtype=c.dtype, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((1, 1), device="cuda")
    call, ask = torch.cuda.Stream(), torch.cuda.Stream()
    fa.device_error()
    torch.cuda.synchronize()
    seen, asked, stop, failed = [0], [0], threading.Event(), []

    def query():
        try:
            while not stop.is_set():
                code = fa.device_error(ask)
                assert code in (0, FA_ERR_PAGE), code
                seen[0] += code == FA_ERR_PAGE
                asked[0] += 1
        except BaseException as e:       # reported below: it would end the thread alone
            failed.append(e)

    thread = threading.Thread(target=query)
    thread.start()
    lost = 0
    for i in range(300):
        before = seen[0]
        if op == "append":
            fa.fa_paged_append(k, k, c.k, c.v, c.table, c.seqlens, stream=call)
        else:
            fa.fa_paged_decode(q, c.k, c.v, c.table, c.seqlens, o, lse, 0.1, stream=call)
        call.synchronize()
        # two whole queries after the call have read the word
        until, limit = asked[0] + 3, time.monotonic() + 10
        while seen[0] == before and asked[0] < until and not failed and time.monotonic() < limit:
            time.sleep(2e-5 * (i % 5))
        lost += seen[0] == before
    stop.set()
    thread.join()
    assert not failed, failed
    assert lost == 0
    assert fa.device_error() == 0
