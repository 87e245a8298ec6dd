"""The 4-bit cache on the GPU: rows quantised and read back, and the decode over
them, each against the float64 oracle (oracle/q4_oracle.py).

The quantiser's units are powers of two, so its bytes have one right value.  Rows
read back are exact but for one rounding to their type (bf16 2^-8, fp16 2^-11 of
the value).  The decode's tolerance is derived at ``check_decode``.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import q4_oracle as O
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


def rng_of(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def i64(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int64))).cuda()


def f64(t):
    return t.double().cpu().numpy()


def rows_of(rng, n, spread=1.0):
    """Rows with dims of different magnitudes, and some rows much larger than others."""
    x = rng.standard_normal((n, 576)) * np.exp(spread * rng.standard_normal(576))
    return x * np.exp2(rng.integers(-3, 4, (n, 1)))


# ---------------------------------------------------------------------------
# Rows into the cache
# ---------------------------------------------------------------------------

def run_append(rng, x, dtype, P, padded=0, pages=None, stream=None, pad_cols=0):
    T = len(x)
    pages = pages or max(2, -(-2 * T // P))
    t = torch.from_numpy(x).to(TYPES[dtype])
    wide = torch.zeros(T, 576 + pad_cols, dtype=t.dtype)
    wide[:, :576] = t
    wide = wide.cuda()
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    if padded:
        slots[rng.permutation(T)[:padded]] = -1
    before = rng.integers(0, 256, (pages * P, O.ROW)).astype(np.uint8)
    cache = torch.from_numpy(before.reshape(pages, P, O.ROW)).cuda()
    mla.mla_quantize_append(wide[:, :512], wide[:, 512:576], i64(slots), cache, check_status=True, stream=stream)
    want = before.copy()
    packed = O.pack(t.double().numpy())
    want[slots[slots >= 0]] = packed[slots >= 0]
    return cache.cpu().numpy().reshape(-1, O.ROW), want


@pytest.mark.parametrize("T, dtype, P, padded, pad_cols", [
    (1, "bf16", 16, 0, 0), (3, "fp32", 64, 1, 0), (64, "bf16", 64, 0, 8), (65, "fp16", 32, 5, 16), (130, "fp32", 16, 17, 4),
    (257, "bf16", 32, 0, 64)])
def test_append_matches_oracle(T, dtype, P, padded, pad_cols):
    rng = rng_of(11, T, P)
    got, want = run_append(rng, rows_of(rng, T, 0.5), dtype, P, padded, pad_cols=pad_cols)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_special_rows(dtype):
    rng = rng_of(12)
    top = float(torch.finfo(TYPES[dtype]).max)
    x = rows_of(rng, 16)
    x[0] = 0
    x[1] = -0.0
    x[2, 7] = math.nan
    x[3, 570] = math.inf
    x[4, 100] = -math.inf
    x[5] = top
    x[6] = np.where(np.arange(576) % 2 == 0, 1.0, -1.0) * 2.0 ** -20      # every value a border of its range
    x[7] = 0
    x[7, 31] = 6 * 2.0 ** 10                                              # one value; the other groups hold zeros
    x[8, :32] *= 2.0 ** 13                                                # groups further below than shifts reach
    x[9] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 72)      # ties
    x[10] = -x[9]
    x[11] = float(torch.finfo(TYPES[dtype]).tiny)
    x[12] = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -130                # subnormal numbers
    x[13] = 1.5                                                           # tops next to 6 * 2^e
    x[14] = 1.5078125
    x[15, 0] = math.nan
    x[15, 1] = math.inf
    got, want = run_append(rng, x, dtype, 16)
    np.testing.assert_array_equal(got, want)


def test_append_reports_a_slot_past_the_cache():
    cache = torch.full((2, 16, 304), 7, dtype=torch.uint8, device="cuda")
    x = torch.ones(3, 576, device="cuda")
    with pytest.raises(mla.MLAError) as e:
        mla.mla_quantize_append(x[:, :512], x[:, 512:], i64([4, 32, -1]), cache, check_status=True)
    assert e.value.status == mla.ERR_DEVICE_BOUNDS
    flat = cache.view(-1, 304).cpu().numpy()
    np.testing.assert_array_equal(flat[4], O.pack_row(np.ones(576)))
    assert (np.delete(flat, 4, 0) == 7).all()
    mla.mla_quantize_append(x[:0, :512], x[:0, 512:], i64([]), cache, check_status=True)     # nothing, and no error left


def test_append_wrapper_checks():
    cache = torch.zeros(2, 16, 304, dtype=torch.uint8, device="cuda")
    x, s = torch.zeros(3, 576, device="cuda"), i64([0, 1, 2])
    for bad, what in (((x[:, :512], x[:, 512:].half(), s, cache), "kpe must be"),
                      ((x[:, :512].double(), x[:, 512:].double(), s, cache), "ckv must be"),
                      ((x[:, :511], x[:, 512:], s, cache), "ckv must be"),
                      ((x[:, :512], x[:2, 512:], s, cache), "kpe must be"),
                      ((x[:, :512], x[:, 512:], s.int(), cache), "slots must be"),
                      ((x[:, :512], x[:, 512:], s, cache[..., :300]), "cache must be"),
                      ((x[:, :512], x[:, 512:], s, cache.view(2, -1)), "cache must be"),
                      ((x[:, :512], x[:, 512:], s, cache.view(torch.int8)), "cache must be"),
                      ((x.t()[:3, :].t()[:, :512], x[:, 512:], s, cache), "ckv must be"),
                      ((x[:, :512].cpu(), x[:, 512:], s, cache), "ckv must be"),
                      ((x[:, 1:513], x[:, 512:], s, cache), None)):
        if what is None:
            with pytest.raises(mla.MLAError):
                mla.mla_quantize_append(*bad)
        else:
            with pytest.raises(ValueError, match=what):
                mla.mla_quantize_append(*bad)


# ---------------------------------------------------------------------------
# Rows out of a cache
# ---------------------------------------------------------------------------

def make_cache(rng, kind, pages, P, kv_scale=1.0):
    """Device cache (two parts or one) and the values it stands for."""
    if kind == "q4":
        b = rng.integers(0, 256, (pages * P, O.ROW)).astype(np.uint8)
        b[:, 288:297] = np.minimum(b[:, 288:297] & 15, 14) | (np.minimum(b[:, 288:297] >> 4, 14) << 4)
        b[:, 297] = rng.integers(127 - 12, 127 + 6, pages * P)
        b[:, 298:] = 0
        return (torch.from_numpy(b.reshape(pages, P, O.ROW)).cuda(), None), O.unpack(b)
    x = torch.from_numpy(rng.standard_normal((pages * P, 576)) * 2)
    x = (x / kv_scale).to(torch.float8_e4m3fn if kind == "fp8" else torch.bfloat16)
    parts = [p.contiguous().view(pages, P, -1).cuda() for p in (x[:, :512], x[:, 512:])]
    return parts, f64(x.float()) * (kv_scale if kind == "fp8" else 1.0)


def page_lists(rng, lens, P, pages):
    counts = [-(-int(n) // P) for n in lens]
    ids = rng.permutation(pages)[:sum(counts)].astype(np.int32)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), ids


def rounded(x, dtype):
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])


@pytest.mark.parametrize("kind", ["q4", "fp8", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lens, P, pad", [([1], 16, 0), ([70, 0, 16, 129, 1, 0], 16, 8), ([33, 64, 200], 32, 0),
                                          ([300, 63, 65, 128], 64, 24)])
def test_read_matches_oracle(kind, dtype, lens, P, pad):
    rng = rng_of(21, len(lens), P)
    pages = sum(-(-n // P) for n in lens) + 3
    scale = 0.25 if kind == "fp8" else 1.0
    (cache, kpe), values = make_cache(rng, kind, pages, P, scale)
    indptr, ids = page_lists(rng, lens, P, pages)
    starts = np.array([rng.integers(0, n + 1) if n > 1 else 0 for n in lens], np.int32)
    starts[0] = 0
    rows = np.concatenate([[0], np.cumsum(np.array(lens) - starts)]).astype(np.int32)
    N = int(rows[-1]) + 4
    ckv = torch.full((N, 512 + pad), 3.0, dtype=TYPES[dtype], device="cuda")
    pe = torch.full((N, 64 + pad), 3.0, dtype=TYPES[dtype], device="cuda")
    mla.mla_read_cache(cache, kpe, i32(indptr), i32(ids), i32(starts), i32(rows), ckv[:, :512], pe[:, :64],
                       kv_scale=scale, check_status=True)
    want = np.full((N, 576), 3.0)
    for r, v in O.read_rows(values, indptr, ids, starts, rows, P):
        want[r] = v
    want = rounded(want, dtype)
    assert torch.equal(ckv[:, :512].cpu(), want[:, :512]) and torch.equal(pe[:, :64].cpu(), want[:, 512:])
    assert (ckv[:, 512:] == 3).all() and (pe[:, 64:] == 3).all()


def test_read_of_special_rows():
    b = np.zeros((16, O.ROW), np.uint8)
    b[:, :288] = 0x77
    b[:, 297] = 127
    b[3, 297] = 255                       # NaN
    b[4, 297] = 127 + 63
    b[5, 297] = 127 - 32
    b[5, 288:297] = 0xee                  # the smallest unit, 2^-46
    cache = torch.from_numpy(b.reshape(1, 16, O.ROW)).cuda()
    for dtype in TYPES:
        ckv = torch.zeros(16, 512, dtype=TYPES[dtype], device="cuda")
        pe = torch.zeros(16, 64, dtype=TYPES[dtype], device="cuda")
        mla.mla_read_cache(cache, None, i32([0, 1]), i32([0]), i32([0]), i32([0, 16]), ckv, pe, check_status=True)
        want = rounded(O.unpack(b), dtype)
        assert torch.equal(ckv.cpu().nan_to_num(9), want[:, :512].nan_to_num(9))
        assert torch.equal(pe.cpu().nan_to_num(9), want[:, 512:].nan_to_num(9))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_read_of_every_unit(dtype):
    """Every exponent with every shift, all eight magnitudes of both signs."""
    rng = rng_of(23)
    b = np.zeros((96 * 15, O.ROW), np.uint8)
    b[:, :288] = rng.integers(0, 256, (len(b), 288))
    first = np.tile(np.arange(15), 96)
    k = (first[:, None] + np.arange(18)) % 15
    b[:, 288:297] = k[:, ::2] | k[:, 1::2] << 4
    b[:, 297] = np.repeat(np.arange(127 - 32, 127 + 64), 15)
    cache = torch.from_numpy(b.reshape(-1, 32, O.ROW)).cuda()
    ckv = torch.zeros(len(b), 512, dtype=TYPES[dtype], device="cuda")
    pe = torch.zeros(len(b), 64, dtype=TYPES[dtype], device="cuda")
    mla.mla_read_cache(cache, None, i32([0, len(b) // 32]), i32(np.arange(len(b) // 32)), i32([0]), i32([0, len(b)]), ckv, pe,
                       check_status=True)
    got, want = torch.cat([ckv, pe], 1).cpu(), rounded(O.unpack(b), dtype)
    assert torch.equal(got, want) and torch.equal(got.signbit(), want.signbit())


def test_read_of_many_requests():
    """4096 requests, most of them without rows."""
    rng = rng_of(22)
    lens = np.zeros(4096, np.int64)
    lens[rng.permutation(4096)[:60]] = rng.integers(1, 40, 60)
    (cache, _), values = make_cache(rng, "q4", 200, 16)
    indptr, ids = page_lists(rng, lens, 16, 200)
    rows = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    N = int(rows[-1])
    ckv, pe = torch.zeros(N, 512, device="cuda"), torch.zeros(N, 64, device="cuda")
    mla.mla_read_cache(cache, None, i32(indptr), i32(ids), i32(np.zeros(4096)), i32(rows), ckv, pe, check_status=True)
    want = np.stack([v for _, v in O.read_rows(values, indptr, ids, np.zeros(4096), rows, 16)])
    np.testing.assert_array_equal(f64(ckv), want[:, :512])
    np.testing.assert_array_equal(f64(pe), want[:, 512:])


@pytest.mark.parametrize("what", ["page", "negative page", "start", "past the list", "list past the array", "rows"])
def test_read_reports_what_it_cannot_reach(what):
    rng = rng_of(23)
    (cache, _), values = make_cache(rng, "q4", 6, 16)
    indptr, ids, starts, rows = np.array([0, 2, 4]), np.array([5, 1, 0, 3]), np.array([0, 0]), np.array([0, 20, 45])
    N, n_idx = 45, 4
    bad = range(0)
    if what == "page":
        ids[1], bad = 6, range(16, 20)
    elif what == "negative page":
        ids[2], bad = -1, range(20, 36)
    elif what == "start":
        starts[1], bad = -3, range(20, 45)
    elif what == "past the list":
        starts[1], bad = 10, range(42, 45)
    elif what == "list past the array":
        n_idx, bad = 3, range(36, 45)
    else:
        N = 40                                        # row_indptr counts 45
    ckv, pe = torch.full((N, 512), 3.0, device="cuda"), torch.full((N, 64), 3.0, device="cuda")
    args = (cache, None, i32(indptr), i32(ids)[:n_idx], i32(starts), i32(rows), ckv, pe)
    with pytest.raises(mla.MLAError) as e:
        mla.mla_read_cache(*args, check_status=True)
    assert e.value.status == mla.ERR_DEVICE_BOUNDS
    got = np.concatenate([f64(ckv), f64(pe)], 1)
    for b in range(2):
        for r in range(rows[b], min(rows[b + 1], N)):
            token = starts[b] + r - rows[b]
            want = np.full(576, 3.0) if r in bad else values[ids[indptr[b] + token // 16] * 16 + token % 16]
            np.testing.assert_array_equal(got[r], want, err_msg=str(r))


def test_read_of_nothing_and_wrapper_checks():
    cache = torch.zeros(2, 16, 304, dtype=torch.uint8, device="cuda")
    ckv, pe = torch.zeros(4, 512, device="cuda"), torch.zeros(4, 64, device="cuda")
    z = i32([0])
    mla.mla_read_cache(cache, None, z, i32([]), i32([]), z, ckv, pe, check_status=True)
    mla.mla_read_cache(cache, None, i32([0, 1]), z, z, i32([0, 0]), ckv[:0], pe[:0], check_status=True)
    ok = [cache, None, i32([0, 1]), z, z, i32([0, 4]), ckv, pe]
    for at, bad, match in ((0, cache[..., :288], "cache must be"), (0, cache.float(), "cache must be"),
                           (1, pe, "cache must be"), (2, i32([0]), "one entry more"),
                           (3, z.long(), "kv_indices must be"), (5, i32([0, 2, 4]), "one entry more"),
                           (6, ckv[:, :511], "ckv_out must be"), (6, ckv.half(), "kpe_out must be"),
                           (7, pe[:3], "kpe_out must be"), (7, pe.cpu(), "kpe_out must be")):
        args = list(ok)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            mla.mla_read_cache(*args)


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------

class Batch:
    """Requests of the given lengths over pages of a pool; `rows` are their values."""

    def __init__(self, rng, lens, H, P, q_len=1, spread=0.3, q_scale=1.0, spare=3, rows=None, poison=True):
        self.rng, self.lens, self.H, self.P, self.q_len = rng, list(lens), H, P, q_len
        self.pages = sum(-(-int(n) // P) for n in lens) + spare
        self.indptr, self.ids = page_lists(rng, lens, P, self.pages)
        x = rows_of(rng, self.pages * P, spread) if rows is None else rows(self.pages * P)
        self.set_rows(x, poison)
        q = torch.from_numpy(rng.standard_normal((len(lens), q_len, H, 576)) * q_scale).to(torch.bfloat16)
        self.set_query(q)
        self.sm_scale = 1 / math.sqrt(192.0)

    def set_query(self, q):
        self.q = q
        shape = (len(self.lens), self.q_len, self.H) if self.q_len > 1 else (len(self.lens), self.H)
        self.q_nope = q[..., :512].reshape(*shape, 512).contiguous().cuda()
        self.q_pe = q[..., 512:].reshape(*shape, 64).contiguous().cuda()

    def set_rows(self, x, poison=True):
        t = torch.from_numpy(np.asarray(x, np.float32)).cuda()
        cache = torch.zeros(self.pages, self.P, 304, dtype=torch.uint8, device="cuda")
        mla.mla_quantize_append(t[:, :512], t[:, 512:], torch.arange(len(t), device="cuda"), cache, check_status=True)
        self.bytes = cache.cpu().numpy().reshape(-1, 304)
        if poison:                        # rows that no request holds: NaN
            held = np.zeros(len(t), bool)
            for b, n in enumerate(self.lens):
                for i in range(-(-int(n) // self.P)):
                    at = self.ids[self.indptr[b] + i] * self.P
                    held[at:at + min(self.P, int(n) - i * self.P)] = True
            self.bytes[~held] = 255
        self.cache = torch.from_numpy(self.bytes.reshape(self.pages, self.P, 304)).cuda()

    def plan(self, dec, **kw):
        dec.plan(self.indptr, i32(self.ids), self.lens, self.P, self.sm_scale, q_len=self.q_len if self.q_len > 1 else 0,
                 **kw)

    def decoder(self):
        dec = mla.MLADecoder(len(self.lens) * self.q_len, self.H, kernel="q4")
        self.plan(dec)
        return dec

    def oracle(self):
        values = np.nan_to_num(O.unpack(self.bytes), nan=0.0)        # NaN rows are not read
        return (values,) + O.decode(f64(self.q), values, self.indptr, self.ids, self.lens, self.P, self.sm_scale,
                                    self.q_len)


def tolerances(b, values, spread):
    """Bounds on the errors of out and lse, element by element.

    Scores: 1152 products (the query in two terms) added in fp32; the errors of
    the additions, 2^-24 of a partial sum each, add up like a random walk, eight
    standard deviations of which are 8 sqrt(1152) 2^-24 < 2^-15.8 of A = sm_scale
    * max_t sum |q_i k_ti|; with the exponential's 2^-22 and the sum's as much
    again: 2^-15 (A + 1).
    Output: p is rounded to fp16 (2^-11 of itself at most) and then held in two
    terms, three and four bits wide: with p in [1, 2) the first leaves a rest of at
    most 2^-3, whose own four bits leave 2^-8.  So p is off by 2^-8 + 2^-11 of
    itself; that and the score's error count twice (numerator and normaliser),
    each relative to the weighted mean of |v|.
    Small p: what the kernel holds is p_t 2^E_t over its largest, G, which is 2^5
    at least; the last term's least unit is 2^-9, so that each is off by up to
    2^-10, 2^-15 G, and those below 2^-17 count as nothing.  Times a value of 6 at
    most: roundings like a random walk of n steps, what is lost n times.  Up to 32
    query rows: from 2^7 down to a unit of 2^-16, 2^-24 G."""
    B, Q, H, _ = b.q.shape
    q = np.abs(f64(b.q))
    A, G, n = np.zeros((B, Q, H)), np.zeros((B, Q, H)), np.zeros((B, 1, 1))
    for i, length in enumerate(b.lens):
        slots = [int(b.ids[b.indptr[i] + t // b.P]) * b.P + t % b.P for t in range(int(length))]
        n[i] = length
        if slots:
            A[i] = (q[i] @ np.abs(values[slots]).T).max(-1) * abs(b.sm_scale)
            s = f64(b.q)[i] @ values[slots].T * b.sm_scale
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            G[i] = (w * 2.0 ** (b.bytes[slots, 297].astype(float) - 127)).max(-1)
            if b.q_len > 1:            # the first query tokens see fewer tokens
                for j in range(Q):
                    seen = int(length) - Q + 1 + j
                    x = np.exp(s[j, :, :seen] - s[j, :, :seen].max(-1, keepdims=True))
                    G[i, j] = (x / x.sum(-1, keepdims=True) * 2.0 ** (b.bytes[slots[:seen], 297].astype(float) - 127)).max(-1)
    lse = 2.0 ** -15 * (A + 1)
    if b.q_len * H > 32:
        small = 5 * np.sqrt(n) * 2.0 ** -15 + n * 2.0 ** -22
    else:
        small = (5 * np.sqrt(n) + n) * 2.0 ** -24
    return (2 * (2.0 ** -8 + 2.0 ** -11) + 2 * lse[..., None]) * spread + (6 * small * G)[..., None] + 1e-30, lse


def check_decode(b, out, lse, what=""):
    values, want, want_lse, spread = b.oracle()
    shape = want.shape
    tol, tol_lse = tolerances(b, values, spread)
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got, got_lse = f64(out).reshape(shape), f64(lse).reshape(shape[:3])
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), what
    assert (got[empty] == 0).all(), what
    worst = np.max(np.abs(got - want) / tol, initial=0)
    worst_lse = np.max(np.abs(got_lse[~empty] - want_lse[~empty]) / tol_lse[~empty], initial=0)
    assert worst <= 1 and worst_lse <= 1, f"{what}: out {worst:.3f}, lse {worst_lse:.3f} of the bound"


def run_check(b, out_dtype=torch.float32, what=""):
    dec = b.decoder()
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=out_dtype)
    dec.check_status()
    check_decode(b, out, lse, what)
    dec.close()
    return out, lse


@pytest.mark.parametrize("H", [1, 4, 16])
@pytest.mark.parametrize("P", [16, 64])
def test_decode_short_lengths(H, P):
    run_check(Batch(rng_of(31, H, P), [1, 0, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65], H, P))


@pytest.mark.parametrize("H", [1, 3, 8, 15, 16, 17, 20, 32, 33, 40, 63, 64, 65, 100, 128])
def test_decode_head_counts(H):
    run_check(Batch(rng_of(32, H), [130, 1, 0, 257], H, 32))


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("H, out_dtype", [(16, torch.bfloat16), (24, torch.float32), (128, torch.bfloat16), (64, torch.float32)])
def test_decode_lengths_around_tiles(P, H, out_dtype):
    run_check(Batch(rng_of(33, P, H), [127, 128, 129, 255, 256, 257, 384, 500], H, P), out_dtype)


@pytest.mark.parametrize("H, lens", [(16, [20000]), (16, [9000, 3, 5000]), (128, [7001]), (40, [6000, 4000]), (1, [12345])])
def test_decode_split_requests(H, lens):
    b = Batch(rng_of(34, H, len(lens)), lens, H, 64)
    dec = b.decoder()
    assert dec.info()["num_partial_slots"] > 1
    dec.close()
    run_check(b)


@pytest.mark.parametrize("H, q_len, lens", [(16, 2, [2, 130, 40, 3]), (16, 4, [4, 127, 128, 131, 700]), (16, 8, [8, 9, 300]),
                                            (32, 4, [129, 260, 5]), (64, 2, [200, 2]), (128, 2, [129, 5]), (20, 3, [128, 3, 64]),
                                            (1, 5, [133, 5]), (48, 3, [140, 3]), (16, 4, [9000, 5])])
def test_decode_several_query_tokens(H, q_len, lens):
    run_check(Batch(rng_of(35, H, q_len), lens, H, 32, q_len=q_len))


@pytest.mark.parametrize("H", [16, 32, 128])
def test_decode_rows_of_different_exponents(H):
    """Rows from 2^-25 to 2^12 side by side, and rows of zeros among them."""
    rng = rng_of(36, H)

    def rows(n):
        x = rng.standard_normal((n, 576)) * np.exp2(rng.integers(-25, 13, (n, 1)).astype(float))
        x[rng.permutation(n)[:n // 8]] = 0
        return x
    b = Batch(rng, [300, 128, 1, 40], H, 64, rows=rows, q_scale=2.0 ** -9)
    run_check(b)


@pytest.mark.parametrize("H", [1, 16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[700, 33], [2500]])
def test_decode_groups_far_apart(H, lens):
    """Every shift up to the largest, in some rows all of them: numbers that are
    subnormal in e4m3 beside such that are not."""
    rng = rng_of(63, H, lens[0])

    def rows(n):
        shift = rng.integers(0, 17, (n, 18))
        shift[rng.permutation(n)[:n // 3]] %= 4
        return rng.standard_normal((n, 576)) * np.repeat(2.0 ** -shift.astype(float), 32, 1)

    b = Batch(rng, lens, H, 32, rows=rows)
    held = b.bytes[b.bytes[:, 297] != 255]
    shifts = np.stack([held[:, 288:297] & 15, held[:, 288:297] >> 4], -1).reshape(len(held), 18)
    assert set(np.unique(shifts)) >= set(range(15))
    run_check(b)


@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_small_rows_weigh_as_much(H):
    """A large row that the query does not look at, beside the small ones it does."""
    rng = rng_of(37, H)

    def rows(n):
        x = rng.standard_normal((n, 576))
        x[:, 0] = 8.0
        x[::7] = 0
        x[::7, 64:128] = 2.0 ** 12
        return x
    b = Batch(rng, [200, 140], H, 32, rows=rows)
    q = np.zeros((2, 1, H, 576))
    q[..., 0] = 20.0 + np.arange(H)
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    run_check(b)


@pytest.mark.parametrize("H", [16, 32, 128])
@pytest.mark.parametrize("gap", [5.0, 11.0, 40.0, 200.0])
@pytest.mark.parametrize("at", [0, 130, 699])
def test_decode_a_token_above_the_rest(H, gap, at):
    """One token `gap` natural units above the others, first, in a later tile or last:
    many small weights are to count where they add up to something."""
    rng = rng_of(38, H, int(gap), at)

    def rows(n):
        x = rng.standard_normal((n, 576)) * 0.5 + 1.0
        x[:, 512:] = 0
        return x
    b = Batch(rng, [700], H, 64, rows=rows)
    values = O.unpack(b.bytes).copy()
    slot = int(b.ids[at // 64]) * 64 + at % 64
    x = np.nan_to_num(values)
    x[:, 512:] = 0
    x[slot, 512] = 4.0
    b.set_rows(x)
    q = np.zeros((1, 1, H, 576))
    q[..., 512] = gap * math.sqrt(192.0) / 4.0
    q[..., 1] = 0.5
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    run_check(b)


@pytest.mark.parametrize("H", [16, 64])
def test_decode_of_a_far_sink_over_a_long_context(H):
    """A token 11.5 natural units above 60000 others, which together weigh most of it."""
    rng = rng_of(39, H)
    n = 60000

    def rows(k):
        x = np.zeros((k, 576))
        x[:, :512] = rng.choice([1.0, 2.0, 3.0], (k, 512))
        return x
    b = Batch(rng, [n], H, 64, rows=rows, poison=False)
    values = O.unpack(b.bytes)
    values[int(b.ids[0]) * 64, 512] = 4.0
    b.set_rows(values, poison=False)
    q = np.zeros((1, 1, H, 576))
    q[..., 512] = 11.5 * math.sqrt(192.0) / 4.0
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    run_check(b)


def test_decode_rising_scores():
    """Every tile's scores above the last one's: the reference moves each time."""
    rng = rng_of(40)
    b = Batch(rng, [1500, 900], 16, 32)
    x = np.nan_to_num(O.unpack(b.bytes))
    for r, n in enumerate(b.lens):
        for t in range(n):
            slot = int(b.ids[b.indptr[r] + t // 32]) * 32 + t % 32
            x[slot, 512:] = 0
            x[slot, 512] = 2.0 ** (t // 128)
    b.set_rows(x)
    q = f64(b.q) * 0.2
    q[..., 512] = 3.0
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    run_check(b)


@pytest.mark.parametrize("H", [16, 128])
def test_decode_nan_rows_and_queries(H):
    b = Batch(rng_of(41, H), [200, 150, 9000], H, 64)
    slot = int(b.ids[b.indptr[1]]) * 64 + 5
    b.bytes[slot, 297] = 255
    b.cache = torch.from_numpy(b.bytes.reshape(b.pages, 64, 304)).cuda()
    b.q_nope[0, 1 % H, 3] = math.nan
    dec = b.decoder()
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert out[0, 1 % H].isnan().all() and lse[0, 1 % H].isnan()
    assert out[2].isfinite().all() and (H == 1 or out[0, 0].isfinite().all())
    dec.close()


def test_decode_large_and_small_queries():
    rng = rng_of(42)
    b = Batch(rng, [300, 77], 16, 32)
    q = f64(b.q) * np.exp2(rng.integers(-12, 3, (2, 1, 16, 1)).astype(float))
    q[0, 0, 3] = 0
    q[0, 0, 4, :512] = 0
    b.set_query(torch.from_numpy(q).to(torch.bfloat16))
    run_check(b)


def test_decode_repeats_bit_for_bit():
    for H, lens in ((16, [9000, 700]), (128, [3000, 100, 64])):
        b = Batch(rng_of(43, H), lens, H, 64)
        dec = b.decoder()
        first = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
        for _ in range(5):
            again = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        rounded_out, _ = dec.run_q4(b.q_nope, b.q_pe, b.cache)
        assert torch.equal(rounded_out, first[0].to(torch.bfloat16))
        dec.check_status()
        dec.close()


@pytest.mark.parametrize("H", [16, 128])
def test_decode_reports_bad_pages(H):
    b = Batch(rng_of(44, H), [200, 100], H, 32)
    dec = b.decoder()
    for bad in (-1, b.pages, 2 ** 31 - 1):
        ids = b.ids.copy()
        ids[2] = bad
        idx = i32(ids)
        dec.plan(b.indptr, idx, b.lens, 32, b.sm_scale)
        out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache)
        with pytest.raises(mla.MLAError) as e:
            dec.check_status()
        assert e.value.status == mla.ERR_DEVICE_BOUNDS
        assert out.isfinite().all()
    b.plan(dec)
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    check_decode(b, out, lse)
    dec.close()


def test_decode_refuses():
    b = Batch(rng_of(45), [40], 16, 32)
    dec = mla.MLADecoder(1, 16, kernel="q4")
    with pytest.raises(mla.MLAError) as e:
        dec.run_q4(b.q_nope, b.q_pe, b.cache)
    assert e.value.status == mla.ERR_NOT_PLANNED
    b.plan(dec)
    bf = torch.zeros(2, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 32, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mla.MLAError) as e:                    # a plan for 4-bit caches does not run another
        dec.run(b.q_nope, b.q_pe, *bf)
    assert e.value.status == mla.ERR_UNSUPPORTED
    other = mla.MLADecoder(1, 16)
    b.plan(other)
    with pytest.raises(mla.MLAError) as e:
        other.run_q4(b.q_nope, b.q_pe, b.cache)
    assert e.value.status == mla.ERR_UNSUPPORTED
    for bad, match in (((b.q_nope, b.q_pe, b.cache[..., :288]), "contiguous"),
                       ((b.q_nope, b.q_pe, b.cache.view(torch.int8)), "cache must be"),
                       ((b.q_nope, b.q_pe, b.cache.view(-1, 16, 304)), "pages of 16"),
                       ((b.q_nope, b.q_pe[..., :32].contiguous(), b.cache), "q_pe"),
                       ((b.q_nope[:, :15].contiguous(), b.q_pe[:, :15].contiguous(), b.cache), "plan's 16 query rows"),
                       ((b.q_nope.float(), b.q_pe, b.cache), "q_pe must have")):
        with pytest.raises(ValueError, match=match):
            dec.run_q4(*bad)
    with pytest.raises(mla.MLAError) as e:
        dec.run_q4(b.q_nope.float(), b.q_pe.float(), b.cache)
    assert e.value.status == mla.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="lse must be float32"):
        dec.run_q4(b.q_nope, b.q_pe, b.cache, lse=torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda"))
    dec.close()
    other.close()


# ---------------------------------------------------------------------------
# Streams, graphs, runs together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H, q_len, lens", [(16, 1, [300, 0, 77]), (128, 1, [5000, 40]), (16, 4, [900, 130])])
def test_rows_behind_the_batch_stay(H, q_len, lens):
    """Buffers for more requests than the plan has: a padded batch."""
    b = Batch(rng_of(58, H, q_len), lens, H, 32, q_len)
    B, more = len(lens), 3
    q_nope, q_pe = (torch.full((B + more, *t.shape[1:]), math.nan, dtype=t.dtype, device="cuda") for t in (b.q_nope, b.q_pe))
    q_nope[:B], q_pe[:B] = b.q_nope, b.q_pe
    out = torch.full(q_nope.shape, 7.0, dtype=torch.float32, device="cuda")
    lse = torch.full(q_nope.shape[:-1], 7.0, dtype=torch.float32, device="cuda")
    dec = mla.MLADecoder((B + more) * q_len, H, kernel="q4")
    b.plan(dec)
    dec.run_q4(q_nope, q_pe, b.cache, out=out, lse=lse)
    dec.check_status()
    check_decode(b, out[:B], lse[:B])
    assert (out[B:] == 7).all() and (lse[B:] == 7).all()
    dec.close()


def test_calls_on_another_stream():
    rng = rng_of(51)
    s = torch.cuda.Stream()
    b = Batch(rng, [200, 31], 16, 32)
    dec = b.decoder()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32, stream=s)
    s.synchronize()
    check_decode(b, out, lse)
    got, want = run_append(rng, rows_of(rng, 70), "bf16", 32, 3, stream=s)
    np.testing.assert_array_equal(got, want)
    dec.close()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages written, read and decoded."""
    rng = rng_of(52)
    P, pages = 64, (1 << 32) // (64 * 304) + 40
    cache = torch.zeros(pages, P, 304, dtype=torch.uint8, device="cuda")
    n = 150
    ids = np.array([pages - 1, 2, pages - 7], np.int32)
    x = rows_of(rng, n, 0.3)
    slots = np.array([ids[t // P] * np.int64(P) + t % P for t in range(n)], np.int64)
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    mla.mla_quantize_append(t[:, :512], t[:, 512:], i64(slots), cache, check_status=True)
    want = O.unpack(O.pack(f64(t)))
    ckv, pe = torch.zeros(n, 512, device="cuda"), torch.zeros(n, 64, device="cuda")
    mla.mla_read_cache(cache, None, i32([0, 3]), i32(ids), i32([0]), i32([0, n]), ckv, pe, check_status=True)
    np.testing.assert_array_equal(np.concatenate([f64(ckv), f64(pe)], 1), want)
    small = Batch(rng, [n], 16, P, rows=lambda k: np.zeros((k, 576)))
    small.ids, small.pages = np.array([0, 1, 2], np.int32), 3
    small.bytes = np.concatenate([O.pack(f64(t)), np.full((3 * P - n, 304), 255, np.uint8)])
    dec = mla.MLADecoder(1, 16, kernel="q4")
    dec.plan([0, 3], i32(ids), [n], P, small.sm_scale)
    out, lse = dec.run_q4(small.q_nope, small.q_pe, cache, out_dtype=torch.float32)
    dec.check_status()
    check_decode(small, out, lse)
    dec.close()


@pytest.mark.parametrize("H, q_len", [(16, 1), (128, 1), (16, 4)])
def test_decode_replayed_after_new_plans(H, q_len):
    rng = rng_of(53, H, q_len)
    b = Batch(rng, [700, 130, 64, 9], H, 32, q_len=q_len)
    dec = b.decoder()
    out = torch.empty(b.q_nope.shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(b.q_nope.shape[:-1], device="cuda")
    idx = i32(np.concatenate([b.ids, np.zeros(64, np.int32)]))
    dec.plan(b.indptr, idx, b.lens, 32, b.sm_scale, q_len=q_len if q_len > 1 else 0)
    dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    for lens in ([700, 130, 64, 9], [300, 50, 60, 5], [20, 100], [max(q_len, 1)] * 4):
        part = Batch.__new__(Batch)
        part.__dict__.update(b.__dict__)
        part.lens = lens
        part.q = b.q[:len(lens)]
        part.indptr = np.concatenate([[0], np.cumsum([-(-n // 32) for n in lens])]).astype(np.int32)
        # the first pages of each request's list
        part.ids = np.concatenate([b.ids[b.indptr[i]:b.indptr[i] + -(-n // 32)] for i, n in enumerate(lens)])
        idx[:len(part.ids)] = i32(part.ids)
        dec.plan(part.indptr, idx, lens, 32, b.sm_scale, q_len=q_len if q_len > 1 else 0)
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        dec.check_status()
        check_decode(part, out[:len(lens)], lse[:len(lens)], str(lens))
        assert (out[len(lens):] == 7).all() and (lse[len(lens):] == 7).all()
    dec.close()


@pytest.mark.parametrize("H", [16, 128])
def test_capture_of_a_plan_without_merges(H):
    """Captured over a plan that splits no request, replayed over one that splits some
    and has an empty one; eager runs of both in between."""
    rng = rng_of(59, H)
    lens = [6000, 40, 0, 33]
    b = Batch(rng, lens, H, 32)
    dec = mla.MLADecoder(len(lens), H, kernel="q4")
    idx = i32(np.concatenate([b.ids, np.zeros(16, np.int32)]))
    small = Batch.__new__(Batch)
    small.__dict__.update(b.__dict__)
    small.lens = [30, 32, 17, 33]
    small.indptr = np.arange(5, dtype=np.int32)
    small.ids = np.concatenate([b.ids[:3], b.ids[b.indptr[3]:b.indptr[3] + 2]])
    small.indptr[4] = 5
    out = torch.empty(b.q_nope.shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(b.q_nope.shape[:-1], device="cuda")

    def plan(part):
        idx[:len(part.ids)] = i32(part.ids)
        dec.plan(part.indptr, idx, part.lens, 32, b.sm_scale)

    def check(part, run, what):
        out.fill_(7.0)
        lse.fill_(7.0)
        run()
        dec.check_status()
        check_decode(part, out, lse, what)

    eager = lambda: dec.run_q4(b.q_nope, b.q_pe, b.cache, out=out, lse=lse)
    plan(small)
    assert dec.info()["num_merge"] == 0
    check(small, eager, "eager, nothing to merge")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eager()
    check(small, g.replay, "replayed, nothing to merge")
    plan(b)
    assert dec.info()["num_merge"] >= 2 and dec.info()["num_partial_slots"] > 1
    check(b, g.replay, "replayed over splits")
    check(b, eager, "eager over splits")
    plan(small)
    check(small, g.replay, "replayed again")
    check(small, eager, "eager again")
    dec.close()


@pytest.mark.parametrize("H, most", [(16, 40), (24, 200), (128, 150)])
def test_decode_of_many_short_requests(H, most):
    """More requests than workers, many of them empty or of one token."""
    rng = rng_of(60, H)
    lens = rng.integers(0, most, 700)
    lens[rng.permutation(700)[:150]] = 0
    lens[rng.permutation(700)[:150]] = 1
    run_check(Batch(rng, lens.tolist(), H, 16), torch.bfloat16)


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("sm_scale", [0.0, -0.05, 2.0])
def test_decode_of_other_scales(H, sm_scale):
    b = Batch(rng_of(61, H), [700, 1, 33, 5000], H, 64, q_scale=0.2)
    b.sm_scale = sm_scale
    run_check(b)


def test_profile_events_around_the_decode():
    b = Batch(rng_of(62), [3000, 20], 16, 64)
    dec = b.decoder()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    stop.record()
    mla.mla_plan_set_profile_events(dec.handle, start, stop)
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    mla.mla_plan_set_profile_events(dec.handle, None, None)
    dec.check_status()
    assert 0 < start.elapsed_time(stop) < 100
    check_decode(b, out, lse)
    dec.close()


def test_a_serving_step_together():
    """Tables, rope append into a bf16 cache of the step's tokens, those rows quantised
    into the pages, the decode over them, and the context read back: captured, and
    replayed for a few steps."""
    rng = rng_of(54)
    B, H, P, pages, maxp = 5, 16, 32, 40, 8
    lens = np.array([0, 31, 64, 100, 5])
    x0 = rows_of(rng, pages * P, 0.3)
    cache = torch.zeros(pages, P, 304, dtype=torch.uint8, device="cuda")
    t0 = torch.from_numpy(x0).to(torch.bfloat16).cuda()
    mla.mla_quantize_append(t0[:, :512], t0[:, 512:], torch.arange(pages * P, device="cuda"), cache)
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, maxp), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-int(n) // P)
        table[b, :k] = ids[at:at + k]
        at += k
    free = np.concatenate([ids[at:], np.full(at, -1, np.int32)])
    d = dict(kv_len=i32(lens), new=i32(np.ones(B)), table=i32(table), free=i32(free), count=i32([pages - at]),
             indptr=i32(np.zeros(B + 1)), indices=i32(np.zeros(B * maxp)), q_indptr=i32(np.zeros(B + 1)),
             slots=i64(np.zeros(B)), pos=i32(np.zeros(B)), status=i32([0]))
    stage = (torch.zeros(1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, 64, dtype=torch.bfloat16, device="cuda"))
    q = torch.zeros(B, H, 576, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    rope = mla.rope_spec(10000.0 ** (-np.arange(32) / 32))
    own_slots = torch.arange(B, device="cuda")
    q_nope, q_pe = torch.zeros(B, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, 64, dtype=torch.bfloat16, device="cuda")
    dec = mla.MLADecoder(B, H, kernel="q4")
    out, lse = torch.zeros(B, H, 512, device="cuda"), torch.zeros(B, H, device="cuda")
    N = B * maxp * P
    rows = i32(np.zeros(B + 1))
    ckv, pe = torch.zeros(N, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 64, dtype=torch.bfloat16, device="cuda")
    zeros = i32(np.zeros(B))

    def step():
        mla.mla_build_tables(d["kv_len"], d["new"], d["table"], d["free"], d["count"], P, d["indptr"], d["indices"],
                             d["q_indptr"], d["slots"], d["pos"], d["status"])
        mla.mla_rope_append(rope, d["pos"], own_slots, q[..., 512:], new[:, :512], new[:, 512:], w, 1e-6, *stage, q_pe_out=q_pe)
        mla.mla_quantize_append(stage[0].view(16, 512)[:B], stage[1].view(16, 64)[:B], d["slots"], cache)
        q_nope.copy_(q[..., :512])
        dec.run_q4(q_nope, q_pe, cache, out=out, lse=lse)
        mla.mla_read_cache(cache, None, d["indptr"], d["indices"], zeros, rows, ckv, pe)

    def plan(n):
        dec.plan(np.concatenate([[0], np.cumsum([-(-int(k) // P) for k in n])]), d["indices"], n, P, 1 / math.sqrt(192.0))
        rows.copy_(i32(np.concatenate([[0], np.cumsum(n)])))

    plan(lens + 1)
    keep = {k: v.clone() for k, v in d.items()}
    kept = cache.clone()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k, v in keep.items():
        d[k].copy_(v)
    cache.copy_(kept)
    for i in range(40):                       # requests grow over their pages' ends
        lens = lens + 1
        plan(lens)
        q.copy_(torch.from_numpy(rng.standard_normal((B, H, 576))))
        new.copy_(torch.from_numpy(rng.standard_normal((B, 576)) * 2))
        before = cache.cpu().numpy().reshape(-1, 304)
        g.replay()
        torch.cuda.synchronize()
        if i % 13 and i < 38:
            continue
        assert int(d["status"]) == 0 and list(d["kv_len"].cpu()) == list(lens)
        slots = d["slots"].cpu().numpy()
        staged = torch.cat([stage[0].view(16, 512)[:B], stage[1].view(16, 64)[:B]], 1)
        want = before.copy()
        want[slots] = O.pack(f64(staged))
        got = cache.cpu().numpy().reshape(-1, 304)
        np.testing.assert_array_equal(got, want)
        b = Batch.__new__(Batch)
        b.lens, b.H, b.P, b.q_len, b.sm_scale = list(lens), H, P, 1, 1 / math.sqrt(192.0)
        b.indptr, b.ids = d["indptr"].cpu().numpy(), d["indices"].cpu().numpy()
        b.bytes, b.q = got, torch.cat([q_nope, q_pe], -1).cpu()[:, None]
        check_decode(b, out, lse, f"step {i}")
        dec.check_status()
        values = O.unpack(got)
        total = int(sum(lens))
        read = np.stack([v for _, v in O.read_rows(values, b.indptr, b.ids, np.zeros(B), rows.cpu().numpy(), P)])
        have = torch.cat([ckv, pe], 1)[:total]
        assert torch.equal(have.cpu(), rounded(read, "bf16"))
        # the plain decode of the rows read back agrees with the decode over the codes
        at = 0
        for r in range(B):
            k = f64(have[at:at + lens[r]])
            at += lens[r]
            s = f64(torch.cat([q_nope, q_pe], -1)[r]) @ k.T / math.sqrt(192.0)
            np.testing.assert_allclose(f64(lse[r]), np.log(np.exp(s - s.max(1, keepdims=True)).sum(1)) + s.max(1), atol=2.0 ** -9)
    dec.close()


@pytest.mark.parametrize("H", [16, 128])
def test_decode_nan_in_a_split_request(H):
    """A NaN row in one share of a request: out and lse of the whole request."""
    b = Batch(rng_of(55, H), [9000, 300], H, 64)
    slot = int(b.ids[b.indptr[0] + 100]) * 64 + 7
    b.bytes[slot, 297] = 255
    b.cache = torch.from_numpy(b.bytes.reshape(b.pages, 64, 304)).cuda()
    dec = b.decoder()
    assert dec.info()["num_partial_slots"] > 1
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isfinite().all() and lse[1].isfinite().all()
    dec.close()


@pytest.mark.parametrize("H, n", [(1, 900), (16, 900), (16, 2000), (40, 1500), (128, 1100)])
def test_decode_nan_in_any_share(H, n):
    """The same with few shares, each of which is read by threads of its own: the row
    at the ends of every tile in turn."""
    b = Batch(rng_of(57, H, n), [n], H, 64)
    dec = b.decoder()
    assert dec.info()["num_partial_slots"] > 1
    for t in sorted({0, n - 1} | set(range(127, n, 128)) | set(range(128, n, 128))):
        slot = int(b.ids[b.indptr[0] + t // 64]) * 64 + t % 64
        flat = b.cache.view(-1, 304)
        was = int(flat[slot, 297])
        flat[slot, 297] = 255
        out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
        assert out.isnan().all() and lse.isnan().all(), t
        flat[slot, 297] = was
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, out_dtype=torch.float32)
    dec.check_status()
    check_decode(b, out, lse)
    dec.close()


@pytest.mark.parametrize("H, lens", [(1, [20000, 0, 150, 9000]), (20, [30000]), (64, [9000] * 4), (100, [5000, 5000]), (128, [12000, 1])])
def test_decode_many_shares(H, lens):
    run_check(Batch(rng_of(56, H), lens, H, 64), torch.bfloat16)


@pytest.mark.parametrize("H, P, k, q_len", [(16, 32, 8, 1), (128, 64, 4, 1), (16, 16, 12, 4)])
def test_sparse_decode_over_a_4bit_cache(H, P, k, q_len):
    """Summaries of the rows read back, the choice of pages, and the decode over them."""
    from oracle import paging_oracle as PO
    rng = rng_of(57, H, P)
    lens = [40 * P - 3, 9 * P, 3 * P + 1, P // 2, 25 * P - 7]
    b = Batch(rng, lens, H, P, q_len=q_len, poison=False)
    n = b.pages * P
    ckv = torch.zeros(b.pages, P, 512, dtype=torch.bfloat16, device="cuda")
    kpe = torch.zeros(b.pages, P, 64, dtype=torch.bfloat16, device="cuda")
    mla.mla_read_cache(b.cache, None, i32([0, b.pages]), torch.arange(b.pages, dtype=torch.int32, device="cuda"), i32([0]),
                       i32([0, n]), ckv.view(n, 512), kpe.view(n, 64), check_status=True)
    summaries = torch.zeros(b.pages, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_summarize_pages(torch.arange(P - 1, n, P, device="cuda"), ckv, kpe, summaries, check_status=True)
    dec = mla.MLASparseDecoder(len(lens) * q_len, H, 64, k, 1, 2, kernel="q4")
    dec.plan(b.indptr, i32(b.ids), lens, P, b.sm_scale, q_len=q_len if q_len > 1 else 0)
    out, lse = dec.run_q4(b.q_nope, b.q_pe, b.cache, summaries, out_dtype=torch.float32)
    dec.check_status()
    # the selected lists, checked against the oracle's choice, then decoded
    sel, ids = dec.sel_indptr.cpu().numpy(), dec.sel_indices.cpu().numpy()
    s64 = f64(summaries)
    for r, count in enumerate(lens):
        pages = b.ids[b.indptr[r]:b.indptr[r + 1]]
        q = f64(b.q)[r].reshape(-1, 576)
        score = (q @ s64[pages].T).max(0)
        got = ids[sel[r]:sel[r + 1]]
        assert len(got) == min(k, len(pages)) and got[-1] == pages[-1] and got[0] == pages[0]
        left = sorted(set(range(1, len(pages) - 2)) - {list(pages).index(p) for p in got}, key=lambda i: -score[i])
        kept = [list(pages).index(p) for p in got]
        inner = [i for i in kept if 1 <= i < len(pages) - 2]
        if left and inner:
            assert min(score[i] for i in inner) >= score[left[0]] - 2.0 ** -10 * abs(score[left[0]])
    part = Batch.__new__(Batch)
    part.__dict__.update(b.__dict__)
    part.lens = [min(k, -(-x // P)) * P - (-x) % P for x in lens]
    part.indptr, part.ids = sel, ids
    check_decode(part, out, lse)
    with pytest.raises(mla.MLAError):                      # the plan is one for 4-bit caches
        dec.run(b.q_nope, b.q_pe, ckv, kpe, summaries)
    dec.close()


def test_two_decoders_and_row_calls_at_once():
    """Decoders of their own on two streams, rows written and read on a third."""
    rng = rng_of(58)
    streams = [torch.cuda.Stream() for _ in range(3)]
    batches = [Batch(rng, [3000, 200, 17], 16, 32), Batch(rng, [900, 1200], 128, 64)]
    decs = [b.decoder() for b in batches]
    x = torch.from_numpy(rows_of(rng, 500)).to(torch.bfloat16).cuda()
    cache = torch.zeros(32, 16, 304, dtype=torch.uint8, device="cuda")
    slots = torch.arange(500, device="cuda")
    ckv, pe = torch.zeros(500, 512, device="cuda"), torch.zeros(500, 64, device="cuda")
    idx, start, rows = torch.arange(32, dtype=torch.int32, device="cuda"), i32([0]), i32([0, 500])
    indptr = i32([0, 32])
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(decs[i].run_q4(batches[i].q_nope, batches[i].q_pe, batches[i].cache, out_dtype=torch.float32,
                                          stream=streams[i]))
        mla.mla_quantize_append(x[:, :512], x[:, 512:], slots, cache, stream=streams[2])
        mla.mla_read_cache(cache, None, indptr, idx, start, rows, ckv, pe, stream=streams[2])
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(batches[i], *outs[i][0])
        for o, l in outs[i][1:]:
            assert torch.equal(o, outs[i][0][0]) and torch.equal(l, outs[i][0][1])
        decs[i].check_status()
        decs[i].close()
    want = O.unpack(O.pack(f64(x)))
    np.testing.assert_array_equal(np.concatenate([f64(ckv), f64(pe)], 1), want)


def test_decode_of_rows_written_out_of_place():
    """Exponents and shifts that no row of mla_quantize_append has: numbers, and no error."""
    rng = rng_of(59)
    for H in (16, 32, 128):
        b = Batch(rng, [300, 40], H, 32)
        b.cache = torch.from_numpy(rng.integers(0, 256, (b.pages, 32, 304)).astype(np.uint8)).cuda()
        dec = b.decoder()
        dec.run_q4(b.q_nope, b.q_pe, b.cache)
        dec.check_status()
        dec.close()
