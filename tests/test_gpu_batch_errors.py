"""What the batch attention's error word says: a wait that gave up and a bad
page table have codes of their own, and each is told alone."""
import ctypes

import pytest
import torch

from .test_gpu_attention_batch import Case, _ints

pytestmark = pytest.mark.gpu

aq = pytest.importorskip("quantized_matmul_affine_gb300")

WAIT, TABLE = 0x0006, 0x0106


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert aq.aq_device_error(clear=True) == 0


@pytest.mark.parametrize("D,members", [(64, 40), (128, 30), (128, 10), (256, 30)])
def test_a_wait_that_gave_up(D, members):
    # the test build (1 ms waits), whose first k tile is not announced
    from quantized_matmul_affine_gb300 import build
    if not build.up_to_date(build.TEST_LIB):
        build.build()
    prod, lib = aq.load(), ctypes.CDLL(build.TEST_LIB)
    for name in ("aq_attention_batch", "aq_attention_batch_workspace_bytes", "aq_device_error"):
        getattr(lib, name).argtypes = getattr(prod, name).argtypes
        getattr(lib, name).restype = getattr(prod, name).restype
    c = Case(10, 2, D, 32, 4, 64, "fp16", 1, [9] * members, [(members, 700)])
    cache = aq.AqCache(torch.from_numpy(c.pool).cuda(), 32, D, 4, 64)
    q, table, lens, starts, shared = c.q.cuda(), *(_ints(x) for x in (c.table, c.lens, c.starts, c.shared))
    n = lib.aq_attention_batch_workspace_bytes(cache._ref, c.B, 1, 10, 1)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    code = ctypes.c_uint32(0)
    told = []
    try:
        for withheld in (3, 0, 3, 0):
            lib.aq_test_withhold(withheld)
            assert lib.aq_attention_batch(
                cache._ref, 0, aq.AQ_F16, q.data_ptr(), 10 * D, table.data_ptr(), lens.data_ptr(),
                starts.data_ptr(), shared.data_ptr(), c.B, 1, 10, 1, table.shape[1], c.scale,
                out.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
            torch.cuda.synchronize()
            assert lib.aq_device_error(ctypes.addressof(code), 1) == 0
            told.append(code.value)
    finally:
        lib.aq_test_withhold(0)
    assert told == [WAIT, 0, WAIT, 0]
    c.check(o=out)


@pytest.mark.parametrize("members", [2, 20])     # 10 and 100 rows a KV head
def test_a_page_outside_the_pool(members):
    c = Case(10, 2, 128, 32, 4, 64, "fp16", 1, [40] * members, [(members, 300)])
    c.table[:, 2] = c.pool.shape[1]
    c.run()
    assert aq.aq_device_error(clear=True) == TABLE
    c.table[:, 2] = -1
    c.run()
    assert aq.aq_device_error(clear=True) == TABLE


def test_groups_that_do_not_ascend():
    c = Case(10, 2, 128, 32, 4, 64, "fp16", 1, [40] * 20, [(20, 300)])
    o = c.run(group_start=_ints([0, 21]))
    assert aq.aq_device_error(clear=True) == TABLE
    c.check(o=o)
