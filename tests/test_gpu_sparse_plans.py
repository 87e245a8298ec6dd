"""Plans of a sparse decoder over its life: captured runs replayed after other
page lists, plans made while the stream is busy, plans that are refused."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

P, H, W = 16, 16, 24


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def indptr_of(lens):
    return np.concatenate([[0], np.cumsum([-(-n // P) for n in lens])]).astype(np.int32)


class World:
    """Caches, summaries and queries of two requests."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

        pages = 2 * W + 5
        self.cc, self.kc = randn(pages, P, 512), randn(pages, P, 64)
        self.summaries = torch.cat([self.cc.float().mean(1), self.kc.float().mean(1)], 1).to(torch.bfloat16)
        self.qn, self.qp = randn(2, H, 512), randn(2, H, 64)
        self.ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.out = torch.zeros((2, H, 512), device="cuda")
        self.lse = torch.zeros((2, H), device="cuda")

    def run(self, dec, stream=None):
        return dec.run(self.qn, self.qp, self.cc, self.kc, self.summaries, self.out, self.lse, stream=stream)

    def expect(self, lens, pages):
        """The run of a decoder that was planned for these lengths alone."""
        dec = mla.MLASparseDecoder(2, H, W, 6, 1, 1)
        try:
            dec.plan(indptr_of(lens), pages, lens, P, 0.07)
            out, lse = dec.run(self.qn, self.qp, self.cc, self.kc, self.summaries, out_dtype=torch.float32)
            dec.check_status()
            return out, lse
        finally:
            dec.close()


@pytest.mark.parametrize("offset", [0, 5])
def test_replay_reads_a_longer_list_than_was_captured(offset):
    """The page list is passed as long as the requests are, and grows at its place between replays."""
    w = World(1)
    lists = w.ids[offset:]
    dec = mla.MLASparseDecoder(2, H, W, 6, 1, 1)

    def plan(lens):
        indptr = indptr_of(lens)
        dec.plan(indptr, lists[:int(indptr[-1])], lens, P, 0.07)

    try:
        plan([100, 37])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.run(dec)
        for lens in ([100, 37], [116, 37], [370, 250], [W * P, W * P], [1, 1], [0, 300]):
            plan(lens)
            w.out.fill_(np.nan)
            g.replay()
            dec.check_status()
            out, lse = w.expect(lens, lists)
            assert torch.equal(w.out, out) and torch.equal(w.lse, lse), lens
    finally:
        dec.close()


def test_plan_does_not_wait_for_the_stream():
    """A plan returns while earlier work of its stream is still running, and the runs queued around it each see
    their own plan."""
    w = World(2)
    side = torch.cuda.Stream()
    dec = mla.MLASparseDecoder(2, H, W, 6, 1, 1)
    first, second = [300, 40], [17, 380]
    try:
        dec.plan(indptr_of(first), w.ids, first, P, 0.07, stream=side)
        with torch.cuda.stream(side):
            w.run(dec)                                   # (loads the kernels)
        torch.cuda.synchronize()
        made = []
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 << 29)                   # some tenths of a second
            busy = torch.cuda.Event()
            busy.record()
            dec.plan(indptr_of(second), w.ids, second, P, 0.07, stream=side)
            assert not busy.query()
            made.append([t.clone() for t in w.run(dec)])
            # (this one may wait for the upload of the plan before it)
            dec.plan(indptr_of(first), w.ids, first, P, 0.07, stream=side)
            made.append([t.clone() for t in w.run(dec)])
        torch.cuda.synchronize()
        dec.check_status()
        for lens, (out, lse) in zip((second, first), made):
            ref, ref_lse = w.expect(lens, w.ids)
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    finally:
        dec.close()


def test_plan_refuses_what_its_runs_would():
    """More requests, or more kept pages, than the scores and the selection take: refused by the plan, which leaves
    the one before it in place."""
    w = World(3)
    dec = mla.MLASparseDecoder(4097, 1, 1, 1, 0, 1)      # (the kept pages of 4097 requests, or of several query tokens each)
    try:
        dec.plan([0, 1], w.ids, [16], P, 0.07)
        with pytest.raises(mla.MLAError) as ei:
            dec.plan(np.zeros(4098, np.int32), w.ids, [0] * 4097, P, 0.07)
        assert ei.value.status == mla.ERR_CAPACITY
        q = torch.zeros((1, 1, 576), dtype=torch.bfloat16, device="cuda")
        out, _ = dec.run(q[..., :512].contiguous(), q[..., 512:].contiguous(), w.cc, w.kc, w.summaries,
                         out_dtype=torch.float32)
        dec.check_status()
        # equal logits: the mean of the page's 16 rows, bf16 probabilities
        ref = w.cc[w.ids[0].long()].double().mean(0)
        assert float((out[0, 0].double() - ref).abs().max()) <= 1e-2
        dec.top_k = 2 ** 30                              # as if it held so many (16 GB)
        with pytest.raises(mla.MLAError) as ei:
            dec.plan([0, 0, 0], w.ids, [0, 0], P, 0.07)
        assert ei.value.status == mla.ERR_CAPACITY
    finally:
        dec.close()
