"""The decode over a 4-bit cache: queries whose dims differ widely, and very large
and very small ones."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from test_gpu_q4 import Batch, f64, rng_of

pytestmark = pytest.mark.gpu


def scores_of_single_tokens(b):
    """lse of requests of one token each, which is the token's score; and the one that
    the oracle has."""
    dec = b.decoder()
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    dec.close()
    values, _, want, _ = b.oracle()
    slots = [int(b.ids[b.indptr[r]]) * b.P for r in range(len(b.lens))]
    return f64(lse).reshape(want.shape), want, values[slots]


@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("ratio", [30.0, 100.0, 300.0, 1000.0])
@pytest.mark.parametrize("dim", [7, 511, 530])
def test_small_dims_beside_a_large_one(H, ratio, dim):
    """One dim `ratio` times the others, keys 0 there.  With the row's largest magnitude
    in [2^7, 2^8) dims down to 2^-7 are held exactly and smaller ones within 2^-15; the
    sums in fp32 are off by 2^-15 of sum |q k| and the rest by as much of 1."""
    rng = rng_of(81, H, int(ratio), dim)

    def rows(n):
        x = rng.standard_normal((n, 576))
        x[:, dim] = 0
        return x
    b = Batch(rng, [1] * 12, H, 16, rows=rows)
    q = f64(b.q)
    q[..., dim] = ratio * np.where(q[..., dim] < 0, -1.0, 1.0)
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    got, want, keys = scores_of_single_tokens(b)
    q = np.abs(f64(b.q))
    up = 2.0 ** (7 - np.floor(np.log2(q.max(-1, keepdims=True))))
    off = np.where(q * up >= 2.0 ** -7, 0.0, np.minimum(q, 2.0 ** -15 / up))
    k = np.abs(keys)[:, None, None, :]
    tol = b.sm_scale * (off * k).sum(-1) + 2.0 ** -15 * (b.sm_scale * (q * k).sum(-1) + 1)
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1, worst


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("q_power, key_power, scale_power", [(115, -30, -90), (120, -20, -105), (-118, 20, 93), (-60, 30, 25),
                                                             (0, -28, 23)])
def test_very_large_and_very_small_queries(H, q_power, key_power, scale_power):
    """Queries to the ends of bf16's range, under scales that make their scores ordinary
    ones: bounds as above, with a largest magnitude of up to 2^5 below [2^7, 2^8)."""
    rng = rng_of(82, H, q_power + 200)
    b = Batch(rng, [1] * 6 + [40], H, 16, rows=lambda n: rng.standard_normal((n, 576)) * 2.0 ** key_power)
    b.sm_scale = 2.0 ** scale_power
    b.set_query(torch.from_numpy(rng.standard_normal((7, 1, H, 576)) * 2.0 ** q_power).to(torch.bfloat16))
    got, want, keys = scores_of_single_tokens(b)
    q, k = np.abs(f64(b.q))[:6], np.abs(keys)[:6, None, None, :]
    off = np.minimum(q, q.max(-1, keepdims=True) * 2.0 ** -18)          # 2^-15 where the largest is 2^3
    tol = b.sm_scale * (off * k).sum(-1) + 2.0 ** -15 * (b.sm_scale * (q * k).sum(-1) + 1)
    worst = np.max(np.abs(got - want)[:6] / tol)
    assert worst <= 1, worst
    assert np.abs(got - want)[6].max() <= 2.0 ** -15 * 64                # sum |q k| of a few times ten
