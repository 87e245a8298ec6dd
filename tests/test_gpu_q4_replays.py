"""Captured decodes over a 4-bit cache, replayed over plans that they were not made for."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import mla
from test_gpu_q4 import Batch, check_decode, i32, rng_of

pytestmark = pytest.mark.gpu


def part_of(b, lens):
    """The first len(lens) requests of a batch, cut to `lens` tokens."""
    part = Batch.__new__(Batch)
    part.__dict__.update(b.__dict__)
    part.lens, part.q = lens, b.q[:len(lens)]
    pages = [-(-n // b.P) for n in lens]
    part.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    part.ids = np.concatenate([b.ids[b.indptr[i]:b.indptr[i] + k] for i, k in enumerate(pages)])
    return part


@pytest.mark.parametrize("H, lens", [(16, [300, 5000, 200, 3000]), (32, [40, 33, 900, 0]), (128, [700, 130, 5000, 64]),
                                     (64, [100] * 4)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_replay_over_a_larger_batch(H, lens, out_dtype):
    """Requests behind the captured ones: their queries are not read, their rows of the
    outputs not written (the arrays here have room for them, so that it shows)."""
    b = Batch(rng_of(95, H, lens[0]), lens, H, 32)
    dec = mla.MLADecoder(4, H, kernel="q4")
    idx = i32(np.concatenate([b.ids, np.zeros(8, np.int32)]))
    out = torch.empty(4, H, 512, dtype=out_dtype, device="cuda")
    lse = torch.empty(4, H, device="cuda")

    def plan(part):
        idx[:len(part.ids)] = i32(part.ids)
        dec.plan(part.indptr, idx, part.lens, 32, b.sm_scale)
        out.fill_(7.0)
        lse.fill_(7.0)

    two = part_of(b, lens[:2])
    plan(two)
    run = lambda: dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    plan(b)
    g.replay()
    dec.check_status()
    check_decode(two, out[:2], lse[:2])
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()
    run()                                     # the call itself takes the batch as planned
    dec.check_status()
    check_decode(b, out, lse)
    plan(two)
    g.replay()
    dec.check_status()
    check_decode(two, out[:2], lse[:2])
    dec.close()


@pytest.mark.parametrize("H, first, other", [(16, 1, 4), (16, 4, 1), (4, 3, 2), (64, 2, 1), (64, 1, 2)])
def test_replay_over_a_plan_of_other_rows(H, first, other):
    """Captured with `first` query tokens that share a pass, replayed over a plan of
    `other`: refused, with the outputs left as they were."""
    b = Batch(rng_of(96, H, first), [300, 5000], H, 32, q_len=first)
    dec = mla.MLADecoder(2 * max(first, other), H, kernel="q4")
    idx = i32(b.ids)
    plan = lambda q: dec.plan(b.indptr, idx, b.lens, 32, b.sm_scale, q_len=q if q > 1 else 0)
    plan(first)
    out = torch.full(b.q_nope.shape, 7.0, device="cuda")
    lse = torch.full(b.q_nope.shape[:-1], 7.0, device="cuda")
    dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    plan(other)
    out.fill_(7.0)
    lse.fill_(7.0)
    g.replay()
    with pytest.raises(mla.MLAError) as e:
        dec.check_status()
    assert e.value.status == mla.ERR_DEVICE_BOUNDS
    assert (out == 7).all() and (lse == 7).all()
    plan(first)
    g.replay()
    dec.check_status()
    check_decode(b, out, lse)
    dec.close()
