"""Float64 CPU oracle for the operators around the decode (page tables, rope
append, page summaries, page scores, page selection).

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``: plain loops over numpy arrays,
written from the definitions in include/mla_paging.h.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def _pi() -> Fraction:
    """Pi to more than 150 digits, by Machin's formula."""
    unit = 10 ** 170

    def arctan_of_inverse(n):
        term, k, total = unit // n, 1, 0
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return Fraction(4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), unit)


PI = _pi()


def build_tables(kv_len, new_len, block_table, free_pages, free_count, page_size, indices_cap, max_tokens):
    """One step with Python lists.  Returns a dict of the arrays after it, or
    the status alone when the step is refused."""
    P = page_size
    table = np.array(block_table)
    num_pages = len(free_pages)
    max_pages = table.shape[1]
    if not 0 <= free_count <= num_pages:
        return dict(status=1)
    stack = [int(p) for p in free_pages[:free_count]]
    held = []
    capacity = False
    for L, n in zip(kv_len, new_len):
        pages = -(-int(L) // P)
        if L < 0 or n < -1 or pages > max_pages:
            return dict(status=1)
        held.append(pages)
    for b, n in enumerate(new_len):
        if n == -1:
            stack += [int(p) for p in table[b, :held[b]]]
    if len(stack) > num_pages:
        return dict(status=1)
    stack_pages = np.array(free_pages)
    lens, indices, indptr, q_indptr, slots, positions = [], [], [0], [0], [], []
    for b, (L, n) in enumerate(zip(kv_len, new_len)):
        L, n = int(L), int(n)
        after = 0 if n < 0 else L + n
        pages = -(-after // P)
        if n >= 0:
            if after > 2 ** 31 - 1 or pages > max_pages:
                return dict(status=3)
            for col in range(held[b], pages):
                if not stack:
                    return dict(status=3)
                table[b, col] = stack.pop()
            for pos in range(L, after):
                slots.append(int(table[b, pos // P]) * P + pos % P)
                positions.append(pos)
            capacity |= len(slots) > max_tokens
        lens.append(after)
        indices += [int(p) for p in table[b, :pages]]
        indptr.append(len(indices))
        q_indptr.append(len(slots))
    if capacity or len(indices) > indices_cap:
        return dict(status=3)
    stack_pages[:len(stack)] = stack
    pad = max_tokens - len(slots)
    return dict(status=0, kv_len=np.array(lens, np.int32), free_count=len(stack), free_pages=stack_pages,
                block_table=table, kv_indptr=np.array(indptr, np.int32), kv_indices=np.array(indices, np.int32),
                q_indptr=np.array(q_indptr, np.int32), slots=np.array(slots + [-1] * pad, np.int64),
                positions=np.array(positions + [0] * pad, np.int32))


def rotate(x, positions, inv_freq, axis_of_pair, interleaved, scale=1.0):
    """x [..., 64] float64 of one token, positions [n_axes] ints -> rotated."""
    out = np.array(x, np.float64)
    for i in range(32):
        # whole turns are taken off the exact product before cos and sin
        turns = int(positions[axis_of_pair[i]]) * Fraction(float(inv_freq[i])) / (2 * PI)
        angle = float((turns - round(turns)) * 2 * PI)
        c, s = scale * np.cos(angle), scale * np.sin(angle)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def norm_row(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def page_mean(ckv_rows, kpe_rows):
    """Rows of one page (float64) -> its 576-wide mean."""
    return np.concatenate([ckv_rows.sum(0), kpe_rows.sum(0)]) / ckv_rows.shape[0]


def page_scores(q, summaries):
    """q [H, 576], summaries [n, 576] float64 -> best score per page."""
    with np.errstate(invalid="ignore"):
        s = summaries @ q.T
    s = np.where(np.isnan(s), -np.inf, s)
    return s.max(1)


def select_pages(scores, pages, top_k, keep_first, keep_last):
    """Page ids kept of one row's list, in its order."""
    n = len(pages)
    if n <= top_k:
        return [int(p) for p in pages]
    kept = set(range(keep_first)) | set(range(n - keep_last, n))
    middle = sorted(range(keep_first, n - keep_last),
                    key=lambda p: (np.inf if np.isnan(scores[p]) else -float(scores[p]), p))
    kept |= set(middle[:top_k - keep_first - keep_last])
    return [int(pages[p]) for p in sorted(kept)]
