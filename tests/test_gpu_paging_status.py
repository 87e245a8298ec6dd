"""Device errors of the operators around the decode: one word for all of them,
which any call's check reads and clears."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


class Calls:
    """Each operator on a cache of four 16-token pages; ``bad`` makes it record an error."""
    names = ("append", "summaries", "scores", "selection")

    def __init__(self):
        self.cache = zeros(4, 16, 512), zeros(4, 16, 64)
        self.summaries = zeros(4, 576)
        self.good, self.past = (torch.tensor([s], dtype=torch.int64, device="cuda") for s in (15, 64))
        self.lists = i32([0, 2]), i32([1, 2])
        self.scores = zeros(1, 2, dtype=torch.float32)
        self.sel = i32([0, 0]), i32([0])
        self.kv = zeros(1, 576)
        self.spec = mla.rope_spec([1.0] * 32)

    def __call__(self, name, bad=False, check=False):
        slots = self.past if bad else self.good
        if name == "append":
            mla.mla_rope_append(self.spec, i32([0]), slots, None, self.kv[:, :512], self.kv[:, 512:], None, 0.0,
                                *self.cache, check_status=check)
        elif name == "summaries":
            mla.mla_summarize_pages(slots, *self.cache, self.summaries, check_status=check)
        elif name == "scores":
            mla.mla_page_scores(zeros(1, 16, 512), zeros(1, 16, 64), self.summaries, self.lists[0],
                                i32([1, 4]) if bad else self.lists[1], self.scores, check_status=check)
        else:
            mla.mla_select_pages(self.scores, i32([0, 3]) if bad else self.lists[0], self.lists[1], 1, 0, 1, *self.sel,
                                 check_status=check)


@pytest.mark.parametrize("wrong", Calls.names)
@pytest.mark.parametrize("asks", Calls.names)
def test_any_check_reports_any_operators_error(wrong, asks):
    call = Calls()
    call("scores", check=True)
    call("append", check=True)
    call(wrong, bad=True)
    with pytest.raises(mla.MLAError) as ei:
        call(asks, check=True)
    assert ei.value.status == mla.ERR_DEVICE_BOUNDS
    for name in Calls.names:                  # and cleared it
        call(name, check=True)


@pytest.mark.parametrize("wrong", Calls.names)
def test_a_sparse_decoders_check_reports_any_operators_error(wrong):
    call = Calls()
    call("scores", check=True)
    call("append", check=True)
    dec = mla.MLASparseDecoder(1, 16, 4, 2)
    try:
        dec.plan([0, 2], call.lists[1], [20], 16, 0.1)
        call(wrong, bad=True)
        dec.run(zeros(1, 16, 512), zeros(1, 16, 64), *call.cache, call.summaries)
        with pytest.raises(mla.MLAError) as ei:
            dec.check_status()
        assert ei.value.status == mla.ERR_DEVICE_BOUNDS
        dec.check_status()
        call("append", check=True)
    finally:
        dec.close()


def test_checks_on_several_streams_at_once():
    """An error is reported once, by one of the checks that run together."""
    import threading
    call = Calls()
    call("scores", check=True)
    call("append", check=True)
    streams = [torch.cuda.Stream() for _ in range(8)]
    empty = torch.zeros(0, dtype=torch.int64, device="cuda")
    for _ in range(20):
        call("append", bad=True)
        torch.cuda.synchronize()
        seen = []

        def ask(stream):
            torch.cuda.set_device(0)
            try:
                mla.mla_summarize_pages(empty, *call.cache, call.summaries, check_status=True, stream=stream)
            except mla.MLAError as e:
                seen.append(e.status)

        threads = [threading.Thread(target=ask, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert seen == [mla.ERR_DEVICE_BOUNDS]


def test_first_calls_of_a_process_are_captured():
    """A capture needs no call before it."""
    import os
    import subprocess
    import sys
    code = """
import torch
import numpy as np
from paged_mla_decode_02_gb300 import mla
z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")
kv, cache, summaries = z(1, 576), (z(4, 16, 512), z(4, 16, 64)), z(4, 576)
kv += 1
slots = torch.tensor([15], device="cuda")
pos, indptr, indices = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0], [0, 2], [1, 0]))
scores, si, sp = z(1, 2, d=torch.float32), z(2, d=torch.int32), z(1, d=torch.int32)
qn, qp = z(1, 16, 512) + 1, z(1, 16, 64) + 1
spec = mla.rope_spec([1.0] * 32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mla.mla_rope_append(spec, pos, slots, None, kv[:, :512], kv[:, 512:], None, 0.0, *cache)
    mla.mla_summarize_pages(slots, *cache, summaries)
    mla.mla_page_scores(qn, qp, summaries, indptr, indices, scores)
    mla.mla_select_pages(scores, indptr, indices, 1, 0, 1, si, sp)
g.replay()
torch.cuda.synchronize()
assert scores.tolist() == [[0.0, 576 / 16]] and si.tolist() == [0, 1] and sp.tolist() == [0]
mla.mla_summarize_pages(slots, *cache, summaries, check_status=True)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
