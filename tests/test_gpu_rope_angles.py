"""The angles of the rotary embedding against exact products of position and
frequency, where fp32 and even fp64 products lose the turn: the ends of the
position range, frequencies above one, tiny and negative ones.

Tolerance.  The kernel's angle is off by less than 2^-31 turns from the fixed
point, and by half a unit in the last place from its rounding to fp32: at most
2^-26 turns, as it lies in [-1/2, 1/2) turns.  Together below 1.01 * 2^-26 *
2 pi = 2^-23.3 radians.  sincospi is good to 2 units in the last place (2^-23
at most, of values up to one), the two products and their sum to 1.5 * 2^-23 of
the pair's magnitude |a| + |b|.  In all less than 2^-21 * (|a| + |b|) before
the rounding to bf16, which adds 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paging_oracle as O
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 12345, 2 ** 20 - 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 129, 2 ** 31 - 4099]


def frequencies(kind):
    i = np.arange(32, dtype=np.float64)
    return {"base 1e4": 10000.0 ** (-i / 32), "base 1e6": 1e6 ** (-i / 32),
            "above one": 10.0 ** (i / 4), "up to 2^40": 2.0 ** (i * 40 / 31) * 1.0,
            "negative": -10.0 ** (i / 4 - 4), "tiny": 10.0 ** (-i)}[kind]


@pytest.mark.parametrize("kind", ["base 1e4", "base 1e6", "above one", "up to 2^40", "negative", "tiny"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_are_exact_to_fp32(kind, interleaved):
    freq = frequencies(kind)
    T = len(POSITIONS)
    rng = np.random.Generator(np.random.PCG64(T))
    q = torch.from_numpy(rng.standard_normal((T, 1, 64)).astype(np.float32)).to(torch.bfloat16)
    kv = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    kv[:, 512:] = q[:, 0].cuda()
    cache = [torch.zeros((1, 16, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64)]
    pos = torch.from_numpy(np.array(POSITIONS, np.int64).astype(np.int32)).cuda()
    out = mla.mla_rope_append(mla.rope_spec(freq, interleaved=interleaved), pos, torch.arange(T, device="cuda"),
                              q.cuda(), kv[:, :512], kv[:, 512:], None, 0.0, *cache, check_status=True)
    got_q, got_k = out[:, 0].double().cpu().numpy(), cache[1][0, :T].double().cpu().numpy()
    x = q[:, 0].double().numpy()
    for t, p in enumerate(POSITIONS):
        ref = O.rotate(x[t], [p], freq, [0] * 32, interleaved)
        pair = np.abs(x[t]).reshape(32, 2).sum(1) if interleaved else np.abs(x[t]).reshape(2, 32).sum(0)
        bound = np.abs(ref) * 2.0 ** -8 + 2.0 ** -21 * (np.repeat(pair, 2) if interleaved else np.tile(pair, 2))
        for got in (got_q, got_k):
            worst = np.argmax(np.abs(got[t] - ref) - bound)
            assert np.all(np.abs(got[t] - ref) <= bound), (p, freq, worst, got[t][worst], ref[worst])
