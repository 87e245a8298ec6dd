"""NaN and infinite products in both forms of the page score kernel (one CTA to
a share of the pages up to 48 heads, a CTA pair above): every head, page and
dim takes part somewhere.  The other values are small whole numbers, whose sums
of products fp32 holds exactly, so the results must be equal to the definition's.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import paging_oracle as O
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 16, 47, 48, 49, 64, 65, 127, 128])
@pytest.mark.parametrize("counts", [[1], [257, 3], [130, 0, 385]])
def test_special_products(heads, counts):
    rng = np.random.Generator(np.random.PCG64([heads, len(counts)]))
    pages = sum(counts) + 3
    q = rng.integers(-2, 3, (len(counts), heads, 576)).astype(np.float64)
    s = rng.integers(-2, 3, (pages, 576)).astype(np.float64)
    # a third of the pages holds an infinity or a NaN somewhere; some heads do
    for p in range(0, pages, 3):
        s[p, rng.integers(576)] = (math.inf, -math.inf, math.nan)[p // 3 % 3]
    for r in range(len(counts)):
        q[r, rng.integers(heads), rng.integers(576)] = math.nan if heads > 1 else 1.0
        if heads > 4:
            q[r, rng.integers(heads), rng.integers(576)] = math.inf
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ids = rng.permutation(pages)[:sum(counts)].astype(np.int32)

    def bf(a):
        return torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda()

    scores = torch.full((len(counts), max(counts)), 9.0, device="cuda")
    mla.mla_page_scores(bf(q[..., :512]).contiguous(), bf(q[..., 512:]).contiguous(), bf(s),
                        torch.from_numpy(indptr).cuda(), torch.from_numpy(ids).cuda(), scores, check_status=True)
    got = scores.cpu().numpy()
    for r, n in enumerate(counts):
        ref = O.page_scores(q[r], s[ids[indptr[r]:indptr[r + 1]]]) if n else np.zeros(0)
        assert np.array_equal(got[r, :n], ref) and np.all(got[r, n:] == 9.0)


@pytest.mark.parametrize("heads", [48, 128])
def test_a_row_of_nan_queries_scores_nothing(heads):
    nan = torch.full((1, heads, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    s = torch.ones((5, 576), dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros((1, 5), device="cuda")
    mla.mla_page_scores(nan[..., :512].contiguous(), nan[..., 512:].contiguous(), s,
                        torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                        torch.arange(5, dtype=torch.int32, device="cuda"), scores, check_status=True)
    assert scores[0].tolist() == [-math.inf] * 5
