"""The latent norm of the append over the whole range of bf16: rows whose squares
fp32 cannot hold, very small or very large, and rows around the border between
the two ways they are summed.

Tolerance: 2^-8 of the value for the rounding to bf16, and 2^-18 for what fp32
adds before (512 squares in pairs of eight and a tree over lanes, below 2^-20;
the root, two products and the powers of two, which are exact, below 2^-21).
An output below the normal range (2^-126) is off by a subnormal step at most.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paging_oracle as O
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

SIZES = [1e-38, 1e-30, 1e-25, 1e-22, 1e-19, 2.0 ** -53, 2.0 ** -50, 2.0 ** -47, 1e-6, 1.0, 1e6, 1e15, 1e17, 4e17, 1e19,
         1e25, 1e37]


def append(rows, weight, eps):
    T = len(rows)
    kv = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    kv[:, :512] = rows
    cache = [torch.zeros((T, 16, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64)]
    mla.mla_rope_append(mla.rope_spec([1.0] * 32), torch.zeros(T, dtype=torch.int32, device="cuda"),
                        torch.arange(T, device="cuda") * 16, None, kv[:, :512], kv[:, 512:], weight, eps, *cache,
                        check_status=True)
    return cache[0][:, 0]


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30, 1e-6, 1e30])
def test_norm_of_small_and_large_rows(eps):
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(len(SIZES), 512, generator=g, dtype=torch.float64) * torch.tensor(SIZES, dtype=torch.float64)[:, None])
    x = x.clamp(-3e38, 3e38).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    got = append(x.cuda(), w.cuda(), eps).double().cpu().numpy()
    eps32 = float(np.float32(eps))
    for i, size in enumerate(SIZES):
        ref = O.norm_row(x[i].double().numpy(), w.double().numpy(), eps32)
        assert np.all(np.abs(got[i] - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133), (size, eps)


def test_norm_of_rows_without_a_finite_one():
    """0 / 0 is NaN where the definition has it; an infinity leaves NaN at its place and 0 elsewhere."""
    x = torch.zeros((3, 512), dtype=torch.bfloat16)
    x[1, 7] = float("inf")
    x[1, 8] = 2.0
    x[2, 3] = float("nan")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    zero, inf, nan = append(x.cuda(), w, 0.0).cpu()
    assert bool(zero.isnan().all()) and bool(nan.isnan().all())
    assert bool(inf[7].isnan()) and inf[8] == 0 and int(inf.isnan().sum()) == 1
    zero, inf, nan = append(x.cuda(), w, 1e-6).cpu()
    assert bool((zero == 0).all()) and bool(nan.isnan().all())
    assert bool(inf[7].isnan()) and inf[8] == 0 and int(inf.isnan().sum()) == 1
