"""Resize on a stream that has only some of the GPU's SMs (a green context of the driver's): its CTAs,
which wait for one another, are no more than run there at once."""
import contextlib
import ctypes
import random

import pytest
import torch

from draft_util import Pool
from test_pool_gpu import books, check_books, int32, shuffled_pool

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def partition(sms):
    """(stream handle, SMs) of a green context with at least `sms` of them."""
    torch.cuda.current_stream().synchronize()          # the primary context is there
    cuda = ctypes.CDLL("libcuda.so.1")
    names = ("cuDeviceGet", "cuDeviceGetDevResource", "cuDevSmResourceSplitByCount",
             "cuDevResourceGenerateDesc", "cuGreenCtxCreate", "cuGreenCtxStreamCreate",
             "cuStreamDestroy_v2", "cuGreenCtxDestroy")
    if not all(hasattr(cuda, n) for n in names):
        pytest.skip("the driver has no green contexts")
    get, resource, split, describe, create, stream_of, end_stream, end = (
        getattr(cuda, n) for n in names)

    def call(fn, *args):
        rc = fn(*args)
        if rc == 801:                                  # CUDA_ERROR_NOT_SUPPORTED
            pytest.skip("green contexts are not supported here")
        assert rc == 0, (fn.__name__, rc)

    class Resource(ctypes.Structure):                  # CUdevResource
        _fields_ = [("type", ctypes.c_int), ("pad", ctypes.c_ubyte * 92),
                    ("sm_count", ctypes.c_uint), ("rest", ctypes.c_ubyte * 44)]

    device, all_sms, some, rest = ctypes.c_int(), Resource(), Resource(), Resource()
    assert ctypes.sizeof(Resource) == 144
    call(get, ctypes.byref(device), torch.cuda.current_device())
    call(resource, device, ctypes.byref(all_sms), 1)   # CU_DEV_RESOURCE_TYPE_SM
    groups = ctypes.c_uint(1)
    call(split, ctypes.byref(some), ctypes.byref(groups), ctypes.byref(all_sms), ctypes.byref(rest),
         ctypes.c_uint(0), ctypes.c_uint(sms))
    desc, ctx, stream = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    call(describe, ctypes.byref(desc), ctypes.byref(some), ctypes.c_uint(1))
    call(create, ctypes.byref(ctx), desc, device, ctypes.c_uint(1))   # CU_GREEN_CTX_DEFAULT_STREAM
    call(stream_of, ctypes.byref(stream), ctx, ctypes.c_uint(1), 0)   # CU_STREAM_NON_BLOCKING
    try:
        yield stream.value, some.sm_count
    finally:
        call(end_stream, stream)
        call(end, ctx)


@pytest.mark.parametrize("B,width", [(40, 4000), (200, 700), (4, 3000), (3, 20)])
def test_resize(B, width):
    """Tables that all SMs, a cluster and one CTA have elsewhere; shared pages are given up at once."""
    import io_aware_attention_fa2_gb300 as fa
    fa.device_error()
    r, page = random.Random(B), 16
    pool = shuffled_pool(r, B * width + 5)
    table = [[-1] * width for _ in range(B)]
    dev, dev_table, granted = books(pool), int32(table), int32([0] * B)
    with partition(16) as (stream, sms):
        assert 16 <= sms < torch.cuda.get_device_properties(0).multi_processor_count

        def resize(dev_t, t, lens, later):
            args = int32(lens), int32(later)
            torch.cuda.synchronize()
            fa.fa_paged_resize(dev, dev_t, *args, granted, page, stream=stream)
            torch.cuda.ExternalStream(stream).synchronize()
            got = pool.resize(t, lens, later, page)
            assert granted.tolist() == got and dev_t.tolist() == t
            check_books(dev, pool)
            return got

        lens = resize(dev_table, table, [0] * B, [r.randint(0, width * page) for _ in range(B)])
        lens = resize(dev_table, table, lens, [r.randint(0, width * page) for _ in range(B)])
        source = [r.randrange(max(1, B // 3)) for _ in range(B)]
        child = fa.paged_fork(dev, dev_table, int32(lens), int32(source), page)
        new, new_lens = pool.fork(table, lens, source, page)[:2]
        torch.cuda.synchronize()
        assert child.seqlens.tolist() == new_lens and -1 not in new_lens
        resize(dev_table, table, lens, [0] * B)
        resize(child.block_table, new, new_lens, [0] * B)
        assert len(pool.free) == len(pool.refs) and isinstance(pool, Pool)
    assert fa.device_error() == 0
