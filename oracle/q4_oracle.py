"""Float64 CPU oracle of the 4-bit latent cache: rows to bytes, bytes to values,
rows read back, and the decode over them.

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``: plain loops over numpy arrays,
written from the definitions in include/mla_decode.h and include/mla_paging.h.
"""
from __future__ import annotations

import math

import numpy as np

ROW, D, GROUP = 304, 576, 32
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def least_exponent(top: float) -> int:
    """The least e with top <= 6 * 2^e (top > 0)."""
    e = math.frexp(top)[1] - 4
    while top > 6 * 2.0 ** e:
        e += 1
    return e


def nearest_code(y: float) -> int:
    """Index of the magnitude nearest to y >= 0, ties to the even index."""
    best = 0
    for i in range(1, 8):
        near, old = abs(MAGNITUDES[i] - y), abs(MAGNITUDES[best] - y)
        if near < old or (near == old and i % 2 == 0):
            best = i
    return best if y < 6 else 7


def pack_row(x) -> np.ndarray:
    """The 304 bytes of a row of 576 values."""
    x = [float(v) for v in x]
    assert len(x) == D
    out = np.zeros(ROW, np.uint8)
    if any(math.isnan(v) for v in x):
        out[297] = 255
        return out
    largest = float(np.finfo(np.float32).max)
    tops = [max(min(abs(v), largest) for v in x[g:g + GROUP]) for g in range(0, D, GROUP)]
    exps = [least_exponent(t) if t > 0 else None for t in tops]
    E = max([e for e in exps if e is not None], default=-32)
    E = min(max(E, -32), 63)
    shifts = [14 if e is None else min(max(E - e, 0), 14) for e in exps]
    for w in range(72):
        word = 0
        for i in range(8):
            v = x[8 * w + i]
            y = min(abs(v), largest) / 2.0 ** (E - shifts[w // 4])
            word |= nearest_code(y) << (4 * i)
            if math.copysign(1.0, v) < 0:
                word |= 1 << (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)
        out[4 * w:4 * w + 4] = [(word >> (8 * b)) & 255 for b in range(4)]
    for g, k in enumerate(shifts):
        out[288 + g // 2] |= k << (4 * (g % 2))
    out[297] = E + 127
    return out


def pack(rows) -> np.ndarray:
    return np.stack([pack_row(r) for r in rows]) if len(rows) else np.zeros((0, ROW), np.uint8)


def unpack(rows) -> np.ndarray:
    """Bytes [n, 304] -> float64 values [n, 576]."""
    rows = np.asarray(rows, np.uint8).reshape(-1, ROW)
    out = np.zeros((len(rows), D))
    words = rows[:, :288].copy().view("<u4").astype(np.int64)
    half = rows[:, 288:297].astype(np.int64)
    table = np.array(MAGNITUDES)
    for d in range(D):
        w, i, g = words[:, d // 8], d % 8, d // GROUP
        sign = (w >> (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)) & 1
        k = (half[:, g // 2] >> (4 * (g % 2))) & 15
        e = rows[:, 297].astype(np.int64) - 127
        out[:, d] = table[(w >> (4 * i)) & 7] * np.where(sign, -1.0, 1.0) * 2.0 ** (e - k)
    out[rows[:, 297] == 255] = np.nan
    return out


def read_rows(values, kv_indptr, kv_indices, starts, row_indptr, page_size):
    """[(row, token's 576 values)] of mla_read_cache; values [num_pages * page_size, 576]."""
    got = []
    for b in range(len(starts)):
        for i in range(int(row_indptr[b + 1]) - int(row_indptr[b])):
            token = int(starts[b]) + i
            page = int(kv_indices[int(kv_indptr[b]) + token // page_size])
            got.append((int(row_indptr[b]) + i, values[page * page_size + token % page_size]))
    return got


def decode(q, values, kv_indptr, kv_indices, kv_len, page_size, sm_scale, q_len=1):
    """q [B, q_len, H, 576], values [num_pages * page_size, 576] -> out [B, q_len,
    H, 512], lse [B, q_len, H], and the softmax-weighted mean of |value|."""
    B, Q, H, _ = q.shape
    out, lse = np.zeros((B, Q, H, 512)), np.full((B, Q, H), -np.inf)
    spread = np.zeros((B, Q, H, 512))
    for b in range(B):
        n = int(kv_len[b])
        slots = [int(kv_indices[int(kv_indptr[b]) + t // page_size]) * page_size + t % page_size for t in range(n)]
        rows = values[slots]
        for j in range(Q):
            seen = rows[:n - q_len + 1 + j]
            if not len(seen):
                continue
            s = (q[b, j] @ seen.T) * sm_scale
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            out[b, j] = p @ seen[:, :512] / total
            spread[b, j] = p @ np.abs(seen[:, :512]) / total
            lse[b, j] = (top + np.log(total))[:, 0]
    return out, lse, spread
