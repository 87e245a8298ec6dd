"""How near the decode over a 4-bit cache comes to the float64 result where the
largest weight says little about it: a token that every query row attends to, of a
value of zero, beside many of random signs whose weights are far below.  What is
compared is the relative L2 error of a request's output in fp32.

Bounds (of weights; the values are on the grid of the cache, so they are exact):
- More than 32 query rows.  A weight in two terms, each to nearest.  The second is
  e5m2 here, off by half of its unit at most, 2^-4 of the rest, that is 2^-7 of the
  power of two in the weight; the error is spread evenly below that in the upper half
  of the rest's range and half as wide in each range below, so its root mean square is
  2^-7 sqrt((1/2 + 1/16 + 1/128 + ..) / 3) = 0.44 * 2^-7 < 2^-8.  Errors of different
  tokens are independent, as the values' signs are: the relative error of the sums is
  that of one weight.  2^-8 in all.
- Up to 32.  fp16's rounding, 2^-11 at most, and of a weight 2^-x of the largest half of
  the last unit 2^-16 where the largest is 2^7: 2^(x - 24) of it.
Both hold for the scores' own errors as well, which are below 2^-13 (scores of a few
units in fp32, and a query that its two terms hold exactly).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import mla
from test_gpu_q4 import Batch, f64, rng_of

pytestmark = pytest.mark.gpu


def grid_rows(rng, n):
    """Rows of the cache's magnitudes with random signs in ckv, zeros in kpe."""
    x = np.zeros((n, 576))
    x[:, :512] = rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], (n, 512)) * rng.choice([-1.0, 1.0], (n, 512))
    return x


def sink_batch(rng, lens, H, P, at, gap, q_len=1, kpe=4.0, spread=0.5):
    """Requests whose token `at` is `gap` natural units above the others (which spread
    by `spread` around 0) and has ckv 0."""
    b = Batch(rng, lens, H, P, q_len=q_len, rows=lambda n: grid_rows(rng, n))
    x = grid_rows(rng, b.pages * P)
    for r, n in enumerate(lens):
        t = min(at, n - 1) if at >= 0 else n - 1
        slot = int(b.ids[b.indptr[r] + t // P]) * P + t % P
        x[slot, :512] = 0
        x[slot, 512] = kpe
    b.set_rows(x)
    q = rng.standard_normal((len(lens), q_len, H, 576))
    q *= spread * math.sqrt(192.0) / math.sqrt(512 * 9.0)      # ckv's mean square is 9.8
    q[..., 512:] = 0
    q[..., 512] = gap * math.sqrt(192.0) / kpe
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    return b


def errors(b):
    """The relative L2 error of each request's output, and the worst of lse."""
    dec = b.decoder()
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    dec.close()
    _, want, want_lse, _ = b.oracle()
    got = f64(out).reshape(want.shape)
    rel = [np.linalg.norm(g - w) / np.linalg.norm(w) for g, w in zip(got, want)]
    return max(rel), np.abs(f64(lse).reshape(want_lse.shape) - want_lse).max()


def bound(rows, powers):
    return 2.0 ** -8 if rows > 32 else 2.0 ** -11 + 2.0 ** (powers - 24)


@pytest.mark.parametrize("H", [16, 32, 33, 64, 128])
@pytest.mark.parametrize("gap", [3.0, 6.0, 8.0, 10.0, 12.0])
@pytest.mark.parametrize("n, at", [(700, 0), (700, 130), (700, 699), (4096, 0), (4096, 2000)])
def test_small_weights_beside_a_large_one(H, gap, n, at):
    rel, lse = errors(sink_batch(rng_of(71, H, int(gap), n, at), [n, n - 63], H, 64, at, gap))
    assert rel <= bound(H, gap / math.log(2)) and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("n", [2, 3, 5, 20, 33, 64, 130])
def test_short_requests_with_a_large_weight(H, n):
    """Few tokens: their errors do not average, and one weight may be off by 2^-7."""
    rel, lse = errors(sink_batch(rng_of(72, H, n), [n, n, n], H, 32, 0, 9.0))
    assert rel <= (2.0 ** -7 if H > 32 else bound(H, 13)) and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H, q_len", [(16, 4), (32, 4), (20, 3)])
def test_several_query_tokens_with_a_large_weight(H, q_len):
    rel, lse = errors(sink_batch(rng_of(73, H, q_len), [700, 1500], H, 32, 0, 9.0, q_len=q_len))
    assert rel <= 2.0 ** -8 and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [16, 64, 128])
def test_a_large_weight_in_a_row_of_a_large_exponent(H):
    """The token's kpe is 2^4 above the others' dims: its row's exponent counts as weight."""
    rel, lse = errors(sink_batch(rng_of(74, H), [900, 3000], H, 64, 0, 7.0, kpe=64.0))
    assert rel <= bound(H, 7 / math.log(2) + 4) and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [64, 128])
def test_large_weights_of_some_rows(H):
    """Half of the query rows see the token far above, the others see it as any other;
    and a request without such a token beside them."""
    rng = rng_of(75, H)
    b = sink_batch(rng, [2000, 900, 1300], H, 64, 0, 9.0)
    q = f64(b.q)
    q[:, :, ::2, 512] = 0
    q[2, ..., 512] = 0
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    rel, lse = errors(b)
    assert rel <= 2.0 ** -8 and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("lens", [[20000, 300], [9000] * 5])
def test_large_weights_in_shares(H, lens):
    """Split requests: one share has the token, the others do not."""
    rel, lse = errors(sink_batch(rng_of(76, H, len(lens)), lens, H, 64, 0, 9.0))
    assert rel <= 2.0 ** -8 and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H, lens", [(16, [4000, 900]), (32, [700]), (64, [4000, 900]), (128, [1200, 130])])
@pytest.mark.parametrize("spread", [0.2, 0.7])
def test_weights_of_like_size(H, lens, spread):
    """No token above the rest: 64 rows hold eight bits of a weight (root mean square
    0.44 * 2^-8), fewer rows as many as fp16."""
    rng = rng_of(77, H)
    b = Batch(rng, lens, H, 64, rows=lambda n: grid_rows(rng, n))
    q = rng.standard_normal((len(lens), 1, H, 576)) * spread * math.sqrt(192.0) / math.sqrt(512 * 9.0)
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    rel, lse = errors(b)
    assert rel <= (2.0 ** -9 if H > 32 else 2.0 ** -11) and lse <= 2.0 ** -12, (rel, lse)


def sinks_batch(rng, n, H, where, gap, more=()):
    """A request whose tokens `where` are `gap` natural units above the others, with ckv 0."""
    b = sink_batch(rng, [n, *more], H, 64, 0, gap)
    values = grid_rows(rng, b.pages * 64)
    for r, length in enumerate(b.lens):
        for t in where:
            if t < length:
                slot = int(b.ids[b.indptr[r] + t // 64]) * 64 + t % 64
                values[slot, :512] = 0
                values[slot, 512] = 4.0
    b.set_rows(values)
    return b


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("where", [range(2), range(4), range(16), range(0, 128, 10), (0, 31, 32, 63, 64, 95, 96, 127)])
def test_several_large_weights(H, where):
    """A few such tokens, adjacent or spread over a tile."""
    rel, lse = errors(sinks_batch(rng_of(80, H, len(where)), 1500, H, where, 9.0, (128, 140, 40)))
    assert rel <= bound(H, 13) and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("at", [0, 500])
def test_either_form_repeats_bit_for_bit(H, at):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = rng_of(81, H, at)
    b = many(sink_batch(rng, [1300], H, 64, at, 9.0), sms if H <= 64 else sms // 2, rng)
    dec = b.decoder()
    first = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    for _ in range(20):
        again = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    dec.check_status()
    dec.close()


def many(b, B, rng):
    """The batch's one request B times over, with other queries: as many as there are CTAs,
    so that none is split and each unit has all its tiles."""
    pages = len(b.ids)
    b.lens = b.lens * B
    b.indptr = (np.arange(B + 1) * pages).astype(np.int32)
    b.ids = np.tile(b.ids, B)
    q = f64(b.q).repeat(B, 0)
    q[..., :512] = q[..., :512][rng.permutation(B)] * rng.choice([-1.0, 1.0], (B, 1, 1, 512))
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    return b


@pytest.mark.parametrize("H", [33, 64, 128])
@pytest.mark.parametrize("gap", [5.0, 8.0, 10.0, 12.0])
@pytest.mark.parametrize("at", [0, 127, 128, 500, 1299])
def test_a_large_weight_in_units_of_many_tiles(H, gap, at):
    """The token in each part of a unit.  Where it is not in the first tile, two tiles go
    by until the other form is taken, with the largest weight at 2^11 and errors of a
    root mean square of 2^-10 / sqrt(3) (a weight 2^-x of the largest: 2^(x - 21.8) of it)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, B = 1300, sms if H <= 64 else sms // 2
    rng = rng_of(78, H, int(gap), at)
    b = many(sink_batch(rng, [n], H, 64, at, gap), B, rng)
    dec = b.decoder()
    assert dec.info()["num_partial_slots"] == 0
    dec.close()
    rel, lse = errors(b)
    late = 2.0 ** (gap / math.log(2) - 21.8) * math.sqrt(256 / n) if at >= 128 else 0.0
    assert rel <= 2.0 ** -8 + late and lse <= 2.0 ** -11, (rel, lse)


@pytest.mark.parametrize("H", [64, 128])
def test_units_that_take_either_form_in_turn(H):
    """Several units to a CTA, with and without such a token: each starts anew."""
    rng = rng_of(79, H)
    B = 400 if H <= 64 else 200
    b = many(sink_batch(rng, [400], H, 64, 70, 9.0), B, rng)
    q = f64(b.q)
    q[rng.permutation(B)[:B // 2], ..., 512] = 0
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    rel, lse = errors(b)
    assert rel <= 2.0 ** -8 and lse <= 2.0 ** -11, (rel, lse)
