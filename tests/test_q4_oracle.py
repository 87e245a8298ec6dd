"""CPU tests of the 4-bit cache: the oracle on rows worked by hand, and the
refusals of the library's entry points, which come before any device work (the
pointers passed here are never followed)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import q4_oracle as O
from paged_mla_decode_02_gb300 import build as B
from paged_mla_decode_02_gb300 import mla


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mla.load_library()


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def row_of(**at):
    x = np.zeros(576)
    for k, v in at.items():
        x[int(k[1:])] = v
    return x


def test_row_worked_example():
    # group 0: top 6 = 6 * 2^0; group 1: top 0.75 = 6 * 2^-3; group 17 (rope): top 48 = 6 * 2^3
    b = O.pack_row(row_of(d0=6, d1=-1, d5=-0.5, d32=0.75, d39=-0.25, d575=48, d574=-4))
    assert b[297] == 3 + 127                               # the row's exponent
    shifts = [(int(b[288 + g // 2]) >> (4 * (g % 2))) & 15 for g in range(18)]
    assert shifts == [3, 6] + [14] * 15 + [0]
    word = lambda w: int.from_bytes(bytes(b[4 * w:4 * w + 4]), "little")
    assert word(0) == 7 | 2 << 4 | 1 << 15 | 1 << 20 | 1 << 11      # 6, -1 (sign bit 15), -0.5 (dim 5: bit 11)
    assert word(4) == 7 | 4 << 28 | 1 << 27                         # 0.75 = 6/8; -0.25 = -2/8 (dim 7: bit 27)
    assert word(71) == 7 << 28 | 1 << 24 | 1 << 19                  # 48 = 6 * 8; -4 = -0.5 * 8 (dim 6: bit 19)
    assert list(b[298:]) == [0] * 6
    got = O.unpack(b[None])[0]
    assert got[0] == 6 and got[1] == -1 and got[5] == -0.5 and got[32] == 0.75 and got[39] == -0.25
    assert got[575] == 48 and got[574] == -4 and not got[64:544].any()


def test_rounding_goes_to_the_even_index():
    for y, code in ((0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5, 6), (5.1, 7), (9, 7)):
        assert O.nearest_code(y) == code, y


def test_special_rows():
    assert O.pack_row(np.zeros(576))[297] == 127 - 32      # the least exponent
    assert not O.unpack(O.pack_row(np.zeros(576))[None]).any()
    nan = O.pack_row(row_of(d3=math.nan, d9=4.0))
    assert nan[297] == 255 and not nan[:297].any() and np.isnan(O.unpack(nan[None])).all()
    inf = O.unpack(O.pack_row(row_of(d3=-math.inf, d9=4.0))[None])[0]
    assert inf[3] == -6 * 2.0 ** 63 and inf[9] == 0
    # a group more than 14 powers of two below the row's
    far = O.unpack(O.pack_row(row_of(d0=6 * 2.0 ** 15, d40=6.0, d41=0.49))[None])[0]
    assert far[40] == 6 and far[41] == 0                   # k = 14: the unit is 2


def test_values_stay_within_half_a_step():
    rng = np.random.Generator(np.random.PCG64(3))
    x = rng.standard_normal((20, 576)) * np.exp(rng.standard_normal((20, 576)))
    got = O.unpack(O.pack(x))
    top = np.abs(x.reshape(20, 18, 32)).max(2, keepdims=True)
    # the unit u is the least with top <= 6 u, so u < top / 3, and the widest step is 2 u
    assert (np.abs(got - x).reshape(20, 18, 32) <= top / 3).all()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

PTR = 1 << 20           # a 16-byte aligned address that no refused call follows


def _quantize(lib, **bad):
    kw = dict(ckv=PTR, cs=512, kpe=PTR, ks=64, dtype=0, slots=PTR, cache=PTR, pages=4, P=16, T=3)
    kw.update(bad)
    return lib.mla_quantize_append(*(kw[k] for k in ("ckv", "cs", "kpe", "ks", "dtype", "slots", "cache", "pages", "P",
                                                     "T")), 0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(ckv=None), mla.ERR_INVALID_ARG), (dict(kpe=None), mla.ERR_INVALID_ARG),
    (dict(slots=None), mla.ERR_INVALID_ARG), (dict(cache=None), mla.ERR_INVALID_ARG),
    (dict(cache=PTR + 8), mla.ERR_INVALID_ARG), (dict(ckv=PTR + 8), mla.ERR_INVALID_ARG),
    (dict(kpe=PTR + 2), mla.ERR_INVALID_ARG), (dict(cs=580), mla.ERR_INVALID_ARG),
    (dict(ks=68), mla.ERR_INVALID_ARG), (dict(dtype=2, cs=514), mla.ERR_INVALID_ARG),
    (dict(pages=0), mla.ERR_INVALID_ARG), (dict(T=-1), mla.ERR_INVALID_ARG), (dict(P=0), mla.ERR_INVALID_ARG),
    (dict(dtype=1), mla.ERR_UNSUPPORTED), (dict(dtype=4), mla.ERR_UNSUPPORTED), (dict(dtype=9), mla.ERR_UNSUPPORTED),
    (dict(P=8), mla.ERR_UNSUPPORTED), (dict(P=128), mla.ERR_UNSUPPORTED), (dict(T=(1 << 24) + 1), mla.ERR_CAPACITY),
])
def test_quantize_refuses(lib, bad, status):
    assert _quantize(lib, **bad) == status


def _read(lib, **bad):
    kw = dict(cache=PTR, kpe=None, dtype=4, scale=1.0, pages=4, P=16, indptr=PTR, indices=PTR, n=9, starts=PTR,
              rows=PTR, batch=2, co=PTR, cs=512, ko=PTR, ks=64, out=0, N=5)
    kw.update(bad)
    return lib.mla_read_cache(*(kw[k] for k in ("cache", "kpe", "dtype", "scale", "pages", "P", "indptr", "indices",
                                                "n", "starts", "rows", "batch", "co", "cs", "ko", "ks", "out", "N")),
                              0, None)


@pytest.mark.parametrize("bad, status", [
    (dict(cache=None), mla.ERR_INVALID_ARG), (dict(cache=PTR + 4), mla.ERR_INVALID_ARG),
    (dict(kpe=PTR), mla.ERR_INVALID_ARG), (dict(dtype=0), mla.ERR_INVALID_ARG),
    (dict(dtype=1, kpe=PTR + 8), mla.ERR_INVALID_ARG), (dict(dtype=1, kpe=PTR, scale=0.0), mla.ERR_INVALID_ARG),
    (dict(dtype=1, kpe=PTR, scale=math.nan), mla.ERR_INVALID_ARG), (dict(indptr=None), mla.ERR_INVALID_ARG),
    (dict(indices=None), mla.ERR_INVALID_ARG), (dict(starts=None), mla.ERR_INVALID_ARG),
    (dict(rows=None), mla.ERR_INVALID_ARG), (dict(co=None), mla.ERR_INVALID_ARG), (dict(ko=None), mla.ERR_INVALID_ARG),
    (dict(co=PTR + 8), mla.ERR_INVALID_ARG), (dict(ko=PTR + 4), mla.ERR_INVALID_ARG),
    (dict(cs=516), mla.ERR_INVALID_ARG), (dict(cs=504), mla.ERR_INVALID_ARG), (dict(ks=56), mla.ERR_INVALID_ARG),
    (dict(out=2, ks=66), mla.ERR_INVALID_ARG), (dict(pages=0), mla.ERR_INVALID_ARG),
    (dict(batch=-1), mla.ERR_INVALID_ARG), (dict(N=-1), mla.ERR_INVALID_ARG), (dict(n=-1), mla.ERR_INVALID_ARG),
    (dict(dtype=2), mla.ERR_UNSUPPORTED), (dict(dtype=3), mla.ERR_UNSUPPORTED), (dict(out=1), mla.ERR_UNSUPPORTED),
    (dict(out=4), mla.ERR_UNSUPPORTED), (dict(P=48), mla.ERR_UNSUPPORTED),
    (dict(batch=4097), mla.ERR_CAPACITY), (dict(N=1 << 31), mla.ERR_CAPACITY),
])
def test_read_refuses(lib, bad, status):
    assert _read(lib, **bad) == status


def test_decode_refuses_a_missing_plan(lib):
    assert lib.mla_decode_run_q4(None, PTR, PTR, 0, PTR, 4, PTR, 0, PTR, None) == mla.ERR_INVALID_ARG


def test_wrapper_refuses_host_tensors():
    q, pe = torch.zeros(1, 16, 512, dtype=torch.bfloat16), torch.zeros(1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q_nope must be a contiguous CUDA tensor"):
        mla.mla_decode_run_q4(None, q, pe, torch.zeros(1, 16, 304, dtype=torch.uint8), q, torch.zeros(1, 16))
