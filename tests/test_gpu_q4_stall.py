"""A wait of the 4-bit decode that runs out, on purpose, in a test build.

The test build (``-DMLA_STALL_TEST``, which the product never loads) limits each
wait to 1 ms and makes one warp of CTA 0 leave out its signal of an expanded
tile.  The warp that issues the scores gives up, the others run out of time or
see that it has, go on without waiting, and the kernel ends by itself; the host
reads MLA_ERR_DEVICE_TIMEOUT, and the next run of the same plan is right.  No
trap, fault or endless loop is involved: every wait has a limit.
"""
from __future__ import annotations

import ctypes
import time

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import build as B
from paged_mla_decode_02_gb300 import mla
from test_gpu_q4 import Batch, check_decode, i32, rng_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def testlib():
    lib = mla.bind_library(B.build_variant("stalltest", ["-DMLA_STALL_TEST"]))
    lib.mla_test_set_q4_stall.restype = ctypes.c_int
    lib.mla_test_set_q4_stall.argtypes = [ctypes.c_int]
    return lib


@pytest.mark.parametrize("H, lens", [(16, [700, 300]), (20, [600, 90]), (128, [900, 200]), (16, [9000, 40])])
@pytest.mark.parametrize("signal", [1, 3])
def test_expired_wait_is_reported_and_leaves_no_state(testlib, H, lens, signal):
    b = Batch(rng_of(61, H, len(lens)), lens, H, 64)
    i32p = ctypes.POINTER(ctypes.c_int32)
    indptr, counts = np.ascontiguousarray(b.indptr, np.int32), np.ascontiguousarray(lens, np.int32)
    ids = i32(b.ids)
    stream = torch.cuda.current_stream().cuda_stream
    h = ctypes.c_void_p()
    # a worker for each request at most, so that CTA 0 has several tiles
    assert testlib.mla_plan_create(len(lens), H, mla.KERNEL_Q4, ctypes.byref(h)) == mla.OK
    assert testlib.mla_decode_plan(h, indptr.ctypes.data_as(i32p), ids.data_ptr(), counts.ctypes.data_as(i32p),
                                   len(lens), H, 512, 64, 64, b.sm_scale, stream) == mla.OK
    info = mla.PlanInfo()
    assert testlib.mla_plan_info(h, ctypes.byref(info)) == mla.OK
    out = torch.empty((len(lens), H, 512), device="cuda")
    lse = torch.empty((len(lens), H), device="cuda")

    def run():
        assert testlib.mla_decode_run_q4(h, b.q_nope.data_ptr(), b.q_pe.data_ptr(), mla.DTYPE_BF16, b.cache.data_ptr(),
                                         b.pages, out.data_ptr(), mla.DTYPE_FP32, lse.data_ptr(), stream) == mla.OK

    try:
        assert testlib.mla_test_set_q4_stall(signal) == 0
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        run()
        status = testlib.mla_plan_check_status(h)
        assert time.perf_counter() - t0 < 5.0               # the kernel ended by itself
        # a unit of one tile has no third signal
        assert status == mla.ERR_DEVICE_TIMEOUT or (signal == 3 and info.total_tiles < 3 * info.num_units and status == mla.OK)
        assert signal == 3 or status == mla.ERR_DEVICE_TIMEOUT
        assert testlib.mla_plan_check_status(h) == mla.OK    # the word was cleared
        assert testlib.mla_test_set_q4_stall(0) == 0
        run()
        assert testlib.mla_plan_check_status(h) == mla.OK
        check_decode(b, out, lse, "after the expired wait")
    finally:
        testlib.mla_test_set_q4_stall(0)
        testlib.mla_plan_destroy(h)
