"""What the calls over a 4-bit cache refuse before they touch the library (no GPU)."""
from __future__ import annotations

import pytest
import torch

from paged_mla_decode_02_gb300 import mla


def decoder(batch, heads, q_len=0):
    """A decoder as plan() leaves it, without a plan of the library's."""
    dec = mla.MLADecoder.__new__(mla.MLADecoder)
    dec.handle, dec.num_heads, dec.page_size, dec.q_len = None, heads, 32, q_len
    dec._rows = batch * max(1, q_len) * heads
    return dec


def queries(*lead):
    return torch.zeros(*lead, 512, dtype=torch.bfloat16), torch.zeros(*lead, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("batch, heads, q_len, lead", [
    (4, 16, 0, (2, 32)),         # as many rows, of other heads
    (4, 16, 0, (1, 64)),
    (4, 16, 0, (64,)),
    (4, 16, 0, (3, 16)),         # too few requests
    (4, 16, 0, (4, 15)),
    (4, 16, 0, (2, 2, 16)),      # query tokens that were not planned
    (4, 16, 0, (1, 4, 1, 16)),
    (4, 16, 2, (2, 4, 16)),
    (4, 16, 2, (3, 32)),
    (4, 16, 2, (4, 16, 2)),
    (4, 16, 2, (3, 2, 16)),
])
def test_queries_of_another_shape_than_planned(batch, heads, q_len, lead):
    with pytest.raises(ValueError, match=f"plan's {batch * max(1, q_len) * heads} query rows as"):
        decoder(batch, heads, q_len).run_q4(*queries(*lead), torch.zeros(2, 32, 304, dtype=torch.uint8))


@pytest.mark.parametrize("batch, heads, q_len, lead", [
    (4, 16, 0, (4, 16)), (4, 16, 0, (7, 16)), (4, 16, 0, (4, 1, 16)), (4, 16, 1, (4, 1, 16)), (4, 16, 1, (4, 16)),
    (4, 16, 2, (4, 2, 16)), (4, 16, 2, (6, 2, 16)), (4, 16, 2, (8, 16)), (4, 16, 2, (4, 32)), (4, 1, 0, (4, 1))])
def test_queries_as_planned_pass_this_check(batch, heads, q_len, lead):
    with pytest.raises(ValueError, match="q_nope must be a contiguous CUDA tensor"):      # the next check's
        decoder(batch, heads, q_len).run_q4(*queries(*lead), torch.zeros(2, 32, 304, dtype=torch.uint8))
