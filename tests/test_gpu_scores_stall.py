"""Waits of the page score kernel that run out, on purpose, in a test build.

The test build (``-DMLA_STALL_TEST``, which the product never loads) limits each
wait to 1 ms and makes one CTA leave out one signal of its page copies, or one
copy of its queries.  The roles that wait for it give up one after the other,
what was issued drains, tensor memory is freed and the kernel returns; the call
reports MLA_ERR_DEVICE_TIMEOUT, and the next one is right.  No trap, fault or
endless loop is involved: every wait has a limit.

The inputs are small whole numbers, so fp32 sums of their products are exact in
any order and the results must be equal to the definition's.
"""
from __future__ import annotations

import ctypes
import time

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import build as B
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

QUERIES = 1000      # from here up the knob names a group of query panels


@pytest.fixture(scope="module")
def testlib():
    lib = mla.bind_library(B.build_variant("stalltest", ["-DMLA_STALL_TEST"]))
    lib.mla_test_set_scores_stall.restype = ctypes.c_int
    lib.mla_test_set_scores_stall.argtypes = [ctypes.c_int]
    return lib


# one CTA a share (16 heads, 7) and CTA pairs (128, 49); the first share has several tiles of a row, or of several
@pytest.mark.parametrize("heads, rows, pages", [(16, 64, 1024), (128, 64, 1024), (7, 500, 200), (49, 500, 200)])
@pytest.mark.parametrize("stall", [1, 2, 9, 12, -1, -4, -11, QUERIES, QUERIES + 2, -QUERIES - 1, -QUERIES - 2])
def test_expired_wait_is_reported_and_leaves_no_state(testlib, heads, rows, pages, stall):
    g = torch.Generator(device="cuda").manual_seed(heads)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.bfloat16)

    summaries, qn, qp = whole(700, 576), whole(rows, heads, 512), whole(rows, heads, 64)
    ids = torch.randint(0, 700, (rows * pages,), generator=g, device="cuda", dtype=torch.int32)
    indptr = torch.arange(rows + 1, device="cuda", dtype=torch.int32) * pages
    scores = torch.zeros((rows, pages), device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        return testlib.mla_page_scores(qn.data_ptr(), qp.data_ptr(), summaries.data_ptr(), 700, indptr.data_ptr(),
                                       ids.data_ptr(), ids.numel(), rows, heads, scores.data_ptr(), pages, pages, 1,
                                       stream)

    try:
        assert testlib.mla_test_set_scores_stall(stall) == 0
        t0 = time.perf_counter()
        assert call() == mla.ERR_DEVICE_TIMEOUT
        assert time.perf_counter() - t0 < 5.0            # the kernel ended by itself
    finally:
        assert testlib.mla_test_set_scores_stall(0) == 0
    scores.fill_(np.nan)
    assert call() == mla.OK
    every = torch.matmul(torch.cat([qn, qp], -1).float(), summaries.float().t()).amax(1)     # [rows, 700], exact
    assert torch.equal(scores, every.gather(1, ids.view(rows, pages).long()))
