"""CPU tests of the paging operators: the oracle on cases worked by hand, and
the refusals of the library's entry points, which come before any device work
(the pointers passed here are never followed)."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

from oracle import paging_oracle as O
from paged_mla_decode_02_gb300 import build as B
from paged_mla_decode_02_gb300 import mla


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mla.load_library()


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def test_tables_worked_example():
    # three requests, pages of 16: one takes its second page, one ends, one stays inside its page
    table = np.array([[7, -1, -1], [3, 5, -1], [9, -1, -1]], np.int32)
    free = np.array([0, 1, 2, -1, -1, -1, -1, -1, -1, -1], np.int32)
    r = O.build_tables([16, 20, 3], [2, -1, 1], table, free, 3, 16, 9, 5)
    assert r["status"] == 0 and list(r["kv_len"]) == [18, 0, 4]
    # pages 3 and 5 went onto the stack, and 5 came off its top
    assert list(r["block_table"][0]) == [7, 5, -1]
    assert r["free_count"] == 4 and list(r["free_pages"][:4]) == [0, 1, 2, 3]
    assert list(r["kv_indptr"]) == [0, 2, 2, 3] and list(r["kv_indices"]) == [7, 5, 9]
    assert list(r["slots"]) == [80, 81, 147, -1, -1] and list(r["positions"]) == [16, 17, 3, 0, 0]
    assert list(r["q_indptr"]) == [0, 2, 2, 3]


def test_tables_refusals_of_the_oracle():
    table, free = np.zeros((1, 2), np.int32), np.array([4, 5, 6], np.int32)
    assert O.build_tables([0], [33], table, free, 3, 16, 9, 99)["status"] == 3      # a third page
    assert O.build_tables([0], [20], table, free, 1, 16, 9, 99)["status"] == 3      # one free page
    assert O.build_tables([0], [20], table, free, 3, 16, 9, 19)["status"] == 3      # 19 token places
    assert O.build_tables([0], [20], table, free, 3, 16, 1, 20)["status"] == 3      # one list entry
    assert O.build_tables([5], [-1], table, free, 3, 16, 9, 9)["status"] == 1       # a fourth page comes back
    assert O.build_tables([-1], [0], table, free, 3, 16, 9, 9)["status"] == 1


def test_rotation_keeps_length_and_follows_its_axis():
    rng = np.random.Generator(np.random.PCG64(1))
    x = rng.standard_normal(64)
    freq = 10000.0 ** (-np.arange(32) / 32)
    axes = [i % 3 for i in range(32)]
    for inter in (True, False):
        y = O.rotate(x, [5, 0, 9], freq, axes, inter)
        assert np.isclose(np.linalg.norm(y), np.linalg.norm(x))
        for i in range(32):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 32)
            if axes[i] == 1:                                   # position 0: not turned
                assert y[a] == x[a] and y[b] == x[b]
        # scores depend on the distance of two positions alone
        z = rng.standard_normal(64)
        one = O.rotate(x, [7, 7, 7], freq, axes, inter) @ O.rotate(z, [3, 3, 3], freq, axes, inter)
        two = O.rotate(x, [104, 104, 104], freq, axes, inter) @ O.rotate(z, [100, 100, 100], freq, axes, inter)
        assert np.isclose(one, two)


def test_selection_worked_example():
    s = np.array([9.0, 1, 5, 5, np.nan, 5, -np.inf, 0])
    pages = [10, 11, 12, 13, 14, 15, 16, 17]
    # ends 0 and 7 kept; the two first of the equal fives
    assert O.select_pages(s, pages, 4, 1, 1) == [10, 12, 13, 17]
    assert O.select_pages(s, pages, 8, 1, 1) == pages
    # NaN and -inf are alike: the lower position first
    assert O.select_pages(s, pages, 7, 1, 1) == [10, 11, 12, 13, 14, 15, 17]


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

PTR = 1 << 20           # a 16-byte aligned address that no refused call follows


def _rope(**bad):
    kw = dict(inv_freq=[1.0] * 32)
    kw.update(bad)
    return mla.rope_spec(**kw)


def _append(lib, rope=None, **bad):
    kw = dict(positions=PTR, axis_stride=0, slots=PTR, q=PTR, qt=128, qh=64, qo=PTR, ckv=PTR, cs=512, kpe=PTR, ks=64,
              w=PTR, eps=1e-6, cc=PTR, kc=PTR, dtype=0, scale=1.0, pages=4, P=16, T=3, H=2)
    kw.update(bad)
    rope = _rope() if rope is None else rope
    return lib.mla_rope_append(ctypes.byref(rope), *(kw[k] for k in (
        "positions", "axis_stride", "slots", "q", "qt", "qh", "qo", "ckv", "cs", "kpe", "ks", "w", "eps", "cc", "kc",
        "dtype", "scale", "pages", "P", "T", "H")), 0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(positions=None), mla.ERR_INVALID_ARG), (dict(slots=None), mla.ERR_INVALID_ARG),
    (dict(q=None), mla.ERR_INVALID_ARG), (dict(qo=None), mla.ERR_INVALID_ARG),
    (dict(ckv=None), mla.ERR_INVALID_ARG), (dict(kpe=None), mla.ERR_INVALID_ARG),
    (dict(cc=None), mla.ERR_INVALID_ARG), (dict(kc=PTR + 8), mla.ERR_INVALID_ARG),
    (dict(q=PTR + 2), mla.ERR_INVALID_ARG), (dict(qo=PTR + 8), mla.ERR_INVALID_ARG),
    (dict(w=PTR + 4), mla.ERR_INVALID_ARG), (dict(cs=580 + 1), mla.ERR_INVALID_ARG),
    (dict(ks=65), mla.ERR_INVALID_ARG), (dict(qt=100), mla.ERR_INVALID_ARG), (dict(qh=68), mla.ERR_INVALID_ARG),
    (dict(eps=-1.0), mla.ERR_INVALID_ARG), (dict(eps=math.nan), mla.ERR_INVALID_ARG),
    (dict(scale=0.0), mla.ERR_INVALID_ARG), (dict(scale=math.inf), mla.ERR_INVALID_ARG),
    (dict(scale=1e-45), mla.ERR_INVALID_ARG), (dict(pages=0), mla.ERR_INVALID_ARG),
    (dict(T=-1), mla.ERR_INVALID_ARG), (dict(H=1025), mla.ERR_INVALID_ARG), (dict(axis_stride=-3), mla.ERR_INVALID_ARG),
    (dict(dtype=2), mla.ERR_UNSUPPORTED), (dict(P=8), mla.ERR_UNSUPPORTED), (dict(P=128), mla.ERR_UNSUPPORTED),
    (dict(T=(1 << 24) + 1), mla.ERR_CAPACITY),
])
def test_append_refuses(lib, bad, status):
    assert _append(lib, **bad) == status


def test_append_refuses_bad_rotations(lib):
    for rope in (_rope(inv_freq=[1.0] * 31 + [math.inf]), _rope(scale=math.nan), _rope(axis_of_pair=[0] * 31 + [8])):
        assert _append(lib, rope) == mla.ERR_INVALID_ARG
    r = _rope(axis_of_pair=[1] * 32)
    r.n_axes = 1                              # pair 0 follows an axis that is not there
    assert _append(lib, r) == mla.ERR_INVALID_ARG
    r.axis_of_pair[:] = [-1] * 32
    assert _append(lib, r) == mla.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        mla.rope_spec([1.0] * 31)


def _tables(lib, **bad):
    kw = dict(kv_len=PTR, new_len=PTR, kv_out=PTR, table=PTR, stride=8, max_pages=8, free=PTR, count=PTR, count_out=PTR,
              num_pages=16, batch=2, P=16, indptr=PTR, indices=PTR, cap=16, q=PTR, slots=PTR, positions=PTR, T=4,
              status=PTR)
    kw.update(bad)
    return lib.mla_build_tables(*kw.values(), None)


@pytest.mark.parametrize("bad, status", [
    (dict(kv_len=None), mla.ERR_INVALID_ARG), (dict(new_len=None), mla.ERR_INVALID_ARG),
    (dict(kv_out=None), mla.ERR_INVALID_ARG), (dict(table=None), mla.ERR_INVALID_ARG),
    (dict(free=None), mla.ERR_INVALID_ARG), (dict(count=None), mla.ERR_INVALID_ARG),
    (dict(count_out=None), mla.ERR_INVALID_ARG), (dict(indptr=None), mla.ERR_INVALID_ARG),
    (dict(indices=None), mla.ERR_INVALID_ARG), (dict(q=None), mla.ERR_INVALID_ARG),
    (dict(slots=None), mla.ERR_INVALID_ARG), (dict(positions=None), mla.ERR_INVALID_ARG),
    (dict(status=None), mla.ERR_INVALID_ARG), (dict(stride=7), mla.ERR_INVALID_ARG),
    (dict(max_pages=0), mla.ERR_INVALID_ARG), (dict(num_pages=0), mla.ERR_INVALID_ARG),
    (dict(batch=-1), mla.ERR_INVALID_ARG), (dict(P=0), mla.ERR_INVALID_ARG), (dict(T=-1), mla.ERR_INVALID_ARG),
    (dict(P=48), mla.ERR_UNSUPPORTED), (dict(batch=4097), mla.ERR_CAPACITY),
    (dict(batch=4096, max_pages=1 << 20, stride=1 << 20), mla.ERR_CAPACITY), (dict(T=1 << 31), mla.ERR_CAPACITY),
])
def test_tables_refuse(lib, bad, status):
    assert _tables(lib, **bad) == status


def _summarize(lib, **bad):
    kw = dict(slots=PTR, T=4, cc=PTR, kc=PTR, dtype=0, scale=1.0, pages=4, P=16, out=PTR)
    kw.update(bad)
    return lib.mla_summarize_pages(*kw.values(), 0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(slots=None), mla.ERR_INVALID_ARG), (dict(out=None), mla.ERR_INVALID_ARG), (dict(T=-1), mla.ERR_INVALID_ARG),
    (dict(out=PTR + 8), mla.ERR_INVALID_ARG), (dict(cc=None), mla.ERR_INVALID_ARG), (dict(P=24), mla.ERR_UNSUPPORTED),
    (dict(dtype=2), mla.ERR_UNSUPPORTED), (dict(scale=-1.0), mla.ERR_INVALID_ARG),
    (dict(T=1 << 25), mla.ERR_CAPACITY),
])
def test_summarize_refuses(lib, bad, status):
    assert _summarize(lib, **bad) == status


def _scores(lib, **bad):
    kw = dict(qn=PTR, qp=PTR, s=PTR, pages=9, indptr=PTR, indices=PTR, n=9, rows=2, H=16, out=PTR, stride=9, most=9)
    kw.update(bad)
    return lib.mla_page_scores(*kw.values(), 0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(qn=None), mla.ERR_INVALID_ARG), (dict(qp=None), mla.ERR_INVALID_ARG), (dict(s=None), mla.ERR_INVALID_ARG),
    (dict(indptr=None), mla.ERR_INVALID_ARG), (dict(indices=None), mla.ERR_INVALID_ARG),
    (dict(out=None), mla.ERR_INVALID_ARG), (dict(qn=PTR + 8), mla.ERR_INVALID_ARG),
    (dict(H=0), mla.ERR_INVALID_ARG), (dict(H=129), mla.ERR_INVALID_ARG), (dict(pages=0), mla.ERR_INVALID_ARG),
    (dict(rows=-1), mla.ERR_INVALID_ARG), (dict(n=-1), mla.ERR_INVALID_ARG), (dict(rows=4097), mla.ERR_CAPACITY),
    (dict(most=10), mla.ERR_INVALID_ARG), (dict(most=-1), mla.ERR_INVALID_ARG),
])
def test_scores_refuse(lib, bad, status):
    assert _scores(lib, **bad) == status


def _select(lib, **bad):
    kw = dict(s=PTR, stride=9, most=9, indptr=PTR, indices=PTR, n=9, rows=2, k=4, kf=1, kl=1, si=PTR, sp=PTR, cap=8)
    kw.update(bad)
    return lib.mla_select_pages(*kw.values(), 0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(s=None), mla.ERR_INVALID_ARG), (dict(indptr=None), mla.ERR_INVALID_ARG),
    (dict(indices=None), mla.ERR_INVALID_ARG), (dict(si=None), mla.ERR_INVALID_ARG),
    (dict(sp=None), mla.ERR_INVALID_ARG), (dict(k=0), mla.ERR_INVALID_ARG), (dict(kf=-1), mla.ERR_INVALID_ARG),
    (dict(kl=0), mla.ERR_INVALID_ARG), (dict(kf=3, kl=2), mla.ERR_INVALID_ARG),
    (dict(kf=2 ** 31 - 1, kl=2 ** 31 - 1, k=2 ** 31 - 1, cap=1 << 40), mla.ERR_INVALID_ARG),
    (dict(cap=7), mla.ERR_CAPACITY), (dict(rows=4097, cap=1 << 20), mla.ERR_CAPACITY),
    (dict(k=2 ** 31 - 1, cap=1 << 40), mla.ERR_CAPACITY),
    (dict(most=10), mla.ERR_INVALID_ARG), (dict(most=-1), mla.ERR_INVALID_ARG),
])
def test_selection_refuses(lib, bad, status):
    assert _select(lib, **bad) == status
