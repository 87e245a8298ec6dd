"""The operators around the decode on the GPU, each against the float64 oracle
(oracle/paging_oracle.py), and a run of them together.

Tolerances.  A result rounded to bf16 is off by at most 2^-8 of its value, to
e4m3 by 2^-4 (2^-10 below the normal range, in units of the scale).  What fp32
adds before the rounding is bounded per test, beside its number.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from gpu_helpers import assert_parity
from oracle import mla_oracle as M
from oracle import paging_oracle as O
from paged_mla_decode_02_gb300 import mla

pytestmark = pytest.mark.gpu

FREQ = 10000.0 ** (-np.arange(32, dtype=np.float64) / 32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


def f64(t):
    return t.double().cpu().numpy()


def rng_of(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


# ---------------------------------------------------------------------------
# Page tables
# ---------------------------------------------------------------------------

def tables_state(rng, lens, P, max_pages, spare, stride=None, caps=None):
    B = len(lens)
    held = [-(-int(n) // P) for n in lens]
    num_pages = sum(held) + spare
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, stride or max_pages), -7, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    free = np.full(num_pages, -5, np.int32)
    free[:spare] = ids[at:]
    return dict(lens=np.asarray(lens, np.int32), table=table, free=free, count=spare, P=P, max_pages=max_pages)


def run_tables(s, new_len, indices_cap, max_tokens, in_place=True, stream=None):
    B = len(s["lens"])
    d = dict(kv_len=i32(s["lens"]), table=dev(s["table"]), free=dev(s["free"]), count=i32([s["count"]]),
             indptr=torch.full((B + 1,), -3, dtype=torch.int32, device="cuda"),
             indices=torch.full((indices_cap,), -3, dtype=torch.int32, device="cuda"),
             q=torch.full((B + 1,), -3, dtype=torch.int32, device="cuda"),
             slots=torch.full((max_tokens,), -3, dtype=torch.int64, device="cuda"),
             positions=torch.full((max_tokens,), -3, dtype=torch.int32, device="cuda"),
             status=torch.full((1,), -3, dtype=torch.int32, device="cuda"))
    d["len_out"] = d["kv_len"] if in_place else torch.full((B,), -3, dtype=torch.int32, device="cuda")
    d["count_out"] = d["count"] if in_place else torch.full((1,), -3, dtype=torch.int32, device="cuda")
    mla.mla_build_tables(d["kv_len"], i32(new_len), d["table"][:, :s["max_pages"]], d["free"], d["count"], s["P"],
                         d["indptr"], d["indices"], d["q"], d["slots"], d["positions"], d["status"],
                         None if in_place else d["len_out"], None if in_place else d["count_out"], stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


def check_tables(s, new_len, indices_cap, max_tokens, in_place=True):
    ref = O.build_tables(s["lens"], new_len, s["table"][:, :s["max_pages"]], s["free"], s["count"], s["P"], indices_cap,
                         max_tokens)
    got = run_tables(s, new_len, indices_cap, max_tokens, in_place)
    assert got["status"][0] == ref["status"]
    if ref["status"]:
        assert np.array_equal(got["len_out"], s["lens"]) and got["count_out"][0] == s["count"]
        assert np.array_equal(got["table"], s["table"]) and np.array_equal(got["free"], s["free"])
        assert np.all(got["slots"] == -1) and np.all(got["positions"] == 0)
        assert np.all(got["indptr"] == -3) and np.all(got["indices"] == -3) and np.all(got["q"] == -3)
        return got
    n = len(ref["kv_indices"])
    assert np.array_equal(got["len_out"], ref["kv_len"]) and got["count_out"][0] == ref["free_count"]
    assert np.array_equal(got["table"][:, :s["max_pages"]], ref["block_table"])
    assert np.array_equal(got["table"][:, s["max_pages"]:], s["table"][:, s["max_pages"]:])
    assert np.array_equal(got["free"], ref["free_pages"])
    assert np.array_equal(got["indptr"], ref["kv_indptr"]) and np.array_equal(got["indices"][:n], ref["kv_indices"])
    assert np.all(got["indices"][n:] == -3)
    assert np.array_equal(got["q"], ref["q_indptr"])
    assert np.array_equal(got["slots"], ref["slots"]) and np.array_equal(got["positions"], ref["positions"])
    if not in_place:
        assert np.array_equal(got["kv_len"], s["lens"]) and got["count"][0] == s["count"]
    return got


@pytest.mark.parametrize("B, P, longest, in_place", [
    (1, 16, 40, True), (2, 64, 1, True), (33, 32, 700, False), (130, 64, 5000, True), (1025, 16, 300, True),
    (4096, 16, 60, False), (3, 16, 60000, True)])
def test_tables_match_oracle(B, P, longest, in_place):
    rng = rng_of(B, P, longest)
    lens = rng.integers(0, longest + 1, B)
    lens[rng.random(B) < 0.15] = 0
    new = rng.integers(0, 4, B)
    new[rng.random(B) < 0.1] = 200
    new[rng.random(B) < 0.2] = -1
    W = (longest + 200) // P + 2
    s = tables_state(rng, lens, P, W, spare=B * (200 // P + 2), stride=W + 3)
    check_tables(s, new, B * W, int(new.clip(0).sum()) + 5, in_place)


def test_tables_corner_steps():
    rng = rng_of(5)
    # nobody does anything; everybody ends; more ends than is taken, and less; a page exactly filled
    s = tables_state(rng, [0, 16, 17, 31, 32], 16, 6, spare=4)
    for new in ([0] * 5, [-1] * 5, [5, -1, -1, 1, 0], [64, -1, 1, 1, 1], [16, 0, 15, 1, 16], [0, 0, -1, 0, 17]):
        check_tables(s, new, 40, 90)
    # nothing to append at all, and no place for it
    check_tables(s, [0, -1, 0, -1, 0], 40, 0)
    # a batch of none
    got = run_tables(dict(s, lens=np.zeros(0, np.int32), table=np.zeros((0, 6), np.int32)), np.zeros(0, np.int32), 4, 3)
    assert got["status"][0] == 0 and got["indptr"][0] == 0 and got["q"][0] == 0 and np.all(got["slots"] == -1)


def test_tables_refused_steps_change_nothing():
    rng = rng_of(6)
    s = tables_state(rng, [0, 16, 17, 31, 32], 16, 6, spare=4)
    new = [20, 1, 0, 2, 16]                                   # 2 + 1 + 0 + 1 + 1 pages, 39 tokens, 12 in all
    check_tables(dict(s, count=3), new, 40, 90)               # five pages wanted
    check_tables(s, [20, 1, 0, 1, 0], 11, 90)                 # fits: 11 list entries
    check_tables(s, [20, 1, 0, 1, 0], 9, 90)
    check_tables(s, [20, 1, 0, 1, 0], 40, 21)
    check_tables(s, [97, 0, 0, 0, 0], 40, 200)                # a row too short
    check_tables(s, [0, -2, 0, 0, 0], 40, 200)
    check_tables(s, [2 ** 31 - 1, 0, 0, 0, 2 ** 31 - 1], 40, 200)
    check_tables(dict(s, lens=np.array([0, -4, 17, 31, 32], np.int32)), [0] * 5, 40, 200)
    check_tables(dict(s, lens=np.array([0, 97, 17, 31, 32], np.int32)), [0] * 5, 40, 200)
    check_tables(dict(s, count=-1), [0] * 5, 40, 200)
    check_tables(dict(s, count=len(s["free"]) + 1), [0] * 5, 40, 200)
    check_tables(dict(s, count=len(s["free"])), [0, 0, 0, 0, -1], 40, 200)


def test_tables_report_bad_page_ids():
    s = tables_state(rng_of(7), [20, 20], 16, 4, spare=3)
    s["table"][1, 1] = len(s["free"])                         # no such page
    got = run_tables(s, [2, 2], 20, 6)
    assert got["status"][0] == mla.ERR_DEVICE_BOUNDS
    assert list(got["len_out"]) == [22, 22] and list(got["slots"][2:]) == [-1] * 4
    assert np.all(got["slots"][:2] == s["table"][0, 1] * 16 + np.array([4, 5]))
    s = tables_state(rng_of(8), [20, 20], 16, 4, spare=3)
    s["free"][2] = -2
    got = run_tables(s, [16, 0], 20, 16)
    assert got["status"][0] == mla.ERR_DEVICE_BOUNDS and np.all(got["slots"][12:] == -1)


def test_tables_of_lists_near_the_largest():
    """16 requests of 2^27 - 1 pages: a page list that ends 16 entries below 2^31,
    the last page of it met by a new token."""
    B, P, most = 16, 16, 2 ** 27 - 1
    n = B * most
    table = torch.arange(n, dtype=torch.int32, device="cuda").bitwise_and_(7).view(B, most)
    kv_len = np.full(B, most * P, np.int32)
    kv_len[-1] -= 1
    new = np.zeros(B, np.int32)
    new[-1] = 1
    indices = torch.full((n + 64,), -3, dtype=torch.int32, device="cuda")
    free, count, status = i32(np.zeros(8)), i32([0]), i32([-3])
    indptr, q, lens = i32(np.full(B + 1, -3)), i32(np.full(B + 1, -3)), i32(kv_len)
    slots, positions = torch.full((1,), -3, dtype=torch.int64, device="cuda"), i32([-3])
    mla.mla_build_tables(lens, i32(new), table, free, count, P, indptr, indices, q, slots, positions, status)
    assert status.item() == 0 and torch.equal(indptr.long().cpu(), torch.arange(B + 1) * most)
    assert torch.equal(indices[:n].view(B, most), table) and bool((indices[n:] == -3).all())
    assert lens.tolist() == [most * P] * B and positions.item() == most * P - 1
    assert slots.item() == table[-1, -1].item() * P + P - 1


def test_tables_replayed_steps():
    """Decode steps in place from one captured graph, against the oracle step by step."""
    rng = rng_of(9)
    lens = rng.integers(0, 90, 37)
    s = tables_state(rng, lens, 16, 12, spare=120)
    B, cap, T = 37, 500, 40
    kv_len, table, free, count = i32(s["lens"]), dev(s["table"]), dev(s["free"]), i32([s["count"]])
    new = i32(np.ones(B))
    o = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, cap, B + 1, T, 1)]
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        mla.mla_build_tables(kv_len, new, table, free, count, 16, o[0], o[1], o[2], slots, o[3], o[4])

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(40):
        n = np.ones(B, np.int64)
        if i % 3 == 1:
            n[rng.integers(0, B)] = -1
        new.copy_(i32(n))
        g.replay()
        ref = O.build_tables(s["lens"], n, s["table"], s["free"], s["count"], 16, cap, T)
        assert ref["status"] == 0 and int(o[4]) == 0
        s.update(lens=ref["kv_len"], table=ref["block_table"], free=ref["free_pages"], count=ref["free_count"])
        assert np.array_equal(kv_len.cpu().numpy(), s["lens"]) and np.array_equal(table.cpu().numpy(), s["table"])
        assert np.array_equal(slots.cpu().numpy(), ref["slots"]) and int(count) == s["count"]
        assert np.array_equal(o[1][:len(ref["kv_indices"])].cpu().numpy(), ref["kv_indices"])


# ---------------------------------------------------------------------------
# Rope append
# ---------------------------------------------------------------------------

def rounded_bound(ref, fp8, kv_scale=1.0):
    """How far a correctly rounded stored value may be from ref (both in real units)."""
    if not fp8:
        return np.abs(ref) * 2.0 ** -8
    return np.maximum(np.abs(ref) * 2.0 ** -4, kv_scale * 2.0 ** -10)


def cache_of(rng, pages, P, fp8):
    def part(w):
        t = torch.from_numpy(rng.standard_normal((pages, P, w)).astype(np.float32))
        return t.to(torch.float8_e4m3fn if fp8 else torch.bfloat16).cuda()
    return part(512), part(64)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("T, H, axes, inter, fp8, P, normed, split", [
    (1, 128, 1, True, False, 64, True, False), (1, 1, 3, False, True, 16, True, True),
    (7, 3, 2, False, False, 32, False, True), (65, 20, 3, True, True, 64, True, False),
    (300, 16, 1, False, True, 32, True, True), (129, 128, 3, False, False, 16, True, True),
    (40, 0, 1, True, False, 64, True, True), (33, 130, 1, True, False, 64, False, False),
    (5, 1024, 2, False, True, 32, True, False), (19, 24, 8, False, False, 64, False, True), (1300, 128, 1, True, False, 64, True, True)])
def test_append_matches_oracle(T, H, axes, inter, fp8, P, normed, split):
    rng = rng_of(T, H, axes)
    pages, scale, kv_scale = T // P + 4, 1.25, 0.3 if fp8 else 1.0
    axis = [i * axes // 32 for i in range(32)] if inter else [i % axes for i in range(32)]
    pos = rng.integers(0, 1 << 20, (axes, T)).astype(np.int32)
    pos[:, 0] = [2 ** 31 - 1, 0, -5, -2 ** 31, 1, 2, 3, 4][:axes]
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    slots[T - 1] = pages * P - 1 if pages * P - 1 not in slots[:-1] else slots[T - 1]
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    q = bf(T, H, 192)[..., 128:] if split else bf(T, H, 64)     # the rope part of a wider query row
    kv = bf(T, 576)
    ckv, kpe = (kv[:, :512], kv[:, 512:]) if split else (kv[:, :512].contiguous(), kv[:, 512:].contiguous())
    w = bf(512) if normed else None
    cc, kc = cache_of(rng, pages, P, fp8)
    before = bits(cc), bits(kc)
    out = torch.full((T, H, 64), 7.0, dtype=torch.bfloat16, device="cuda") if H else None
    rope = mla.rope_spec(FREQ, axis, inter, scale)
    mla.mla_rope_append(rope, dev(pos), dev(slots), q if H else None, ckv, kpe, w, 1e-5, cc, kc, q_pe_out=out,
                        kv_scale=kv_scale, check_status=True)
    got_c, got_k = f64(cc.float()).reshape(-1, 512) * kv_scale, f64(kc.float()).reshape(-1, 64) * kv_scale
    untouched = np.ones(pages * P, bool)
    untouched[slots[slots >= 0]] = False
    eb = 1 if fp8 else 2
    assert np.array_equal(bits(cc).reshape(-1, 512 * eb)[untouched], before[0].reshape(-1, 512 * eb)[untouched])
    assert np.array_equal(bits(kc).reshape(-1, 64 * eb)[untouched], before[1].reshape(-1, 64 * eb)[untouched])
    for t in range(T):
        if slots[t] < 0:
            if H:
                assert bool((out[t] == 7.0).all())
            continue
        # fp32: the angle is off by pi 2^-25 at most, sincospi by 2 units of 2^-24, the products and the sum by
        # 3 x 2^-24 and the scale by 2^-24 of |a| + |b|: less than 2^-20 of it in all; 1 / kv_scale adds 2^-23
        for x, got, f8 in ([(f64(q[t]), f64(out[t]), False)] if H else []) + [(f64(kpe[t]), got_k[slots[t]], fp8)]:
            ref = O.rotate(x, pos[:, t], FREQ, axis, inter, scale)
            if f8:
                ref = np.clip(ref, -448 * kv_scale, 448 * kv_scale)
            both = np.abs(x).max(-1, keepdims=True) * 2 * scale
            assert np.all(np.abs(got - ref) <= rounded_bound(ref, f8, kv_scale) + both * 2.0 ** -20), t
        # the sum of 512 squares in fp32: 21 additions deep, halved by the root; rsqrt 2, three products 3: < 2^-19
        ref = O.norm_row(f64(ckv[t]), f64(w) if normed else None, 1e-5)
        if fp8:
            ref = np.clip(ref, -448 * kv_scale, 448 * kv_scale)
        assert np.all(np.abs(got_c[slots[t]] - ref) <= rounded_bound(ref, fp8, kv_scale) + np.abs(ref) * 2.0 ** -18), t


def test_append_in_place_and_equal_axes():
    """q rotated in place, and text positions expanded over three axes: the bits of the plain call."""
    rng = rng_of(31)
    T, H = 21, 16
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    q, kv = bf(T, H, 64), bf(T, 576)
    pos, slots = i32(rng.integers(0, 9000, T)), dev(rng.permutation(64)[:T].astype(np.int64))
    caches = [cache_of(rng_of(1), 4, 16, False) for _ in range(2)]
    one = mla.mla_rope_append(mla.rope_spec(FREQ), pos, slots, q, kv[:, :512], kv[:, 512:], None, 0.0, *caches[0])
    three = mla.rope_spec(FREQ, [i % 3 for i in range(32)])
    mla.mla_rope_append(three, pos[None].expand(3, T), slots, q, kv[:, :512], kv[:, 512:], None, 0.0, *caches[1],
                        q_pe_out=q, check_status=True)
    assert torch.equal(q, one) and torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_special_values(fp8):
    """Infinities saturate (e4m3) or stay, NaN stays in its own row, zero rows stay zero under a norm."""
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((3, 576), dtype=torch.bfloat16, device="cuda")
    kv[1, 5], kv[1, 512] = math.inf, 1000.0
    kv[2, 7] = math.nan
    cc, kc = cache_of(rng_of(2), 1, 16, fp8)
    slots = dev(np.array([3, 4, 5], np.int64))
    zero = i32(np.zeros(3))
    mla.mla_rope_append(mla.rope_spec(FREQ), zero, slots, q, kv[:, :512], kv[:, 512:], None, 0.0, cc, kc,
                        check_status=True)
    c, k = cc.float()[0].cpu(), kc.float()[0].cpu()
    assert bool((c[3] == 0).all()) and bool((k[3] == 0).all())
    assert c[4, 5] == (448 if fp8 else math.inf) and k[4, 0] == (448 if fp8 else 1000)
    assert bool(c[5, 7].isnan()) and int(c.isnan().sum()) == 1 and int(k.isnan().sum()) == 0
    one = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    mla.mla_rope_append(mla.rope_spec(FREQ), zero, slots, None, kv[:, :512], kv[:, 512:], one, 1e-6, cc, kc,
                        check_status=True)
    assert bool((cc.float()[0, 3] == 0).all()) and bool(cc.float()[0, 5].isnan().all())


def test_append_reports_a_slot_past_the_cache():
    rng = rng_of(3)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    q, kv = bf(2, 4, 64), bf(2, 576)
    cc, kc = cache_of(rng, 2, 16, False)
    before = cc.clone(), kc.clone()
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (mla.rope_spec(FREQ), i32([1, 2]), dev(np.array([32, -1], np.int64)), q, kv[:, :512], kv[:, 512:], None, 0.0,
            cc, kc)
    with pytest.raises(mla.MLAError) as ei:
        mla.mla_rope_append(*args, q_pe_out=out, check_status=True)
    assert ei.value.status == mla.ERR_DEVICE_BOUNDS
    assert torch.equal(cc, before[0]) and torch.equal(kc, before[1]) and bool((out == 7.0).all())
    args[2].fill_(-1)
    mla.mla_rope_append(*args, q_pe_out=out, check_status=True)          # the report was cleared


def test_append_of_nothing():
    cc, kc = cache_of(rng_of(4), 1, 16, False)
    e = torch.empty((0, 576), dtype=torch.bfloat16, device="cuda")
    out = mla.mla_rope_append(mla.rope_spec(FREQ), i32([]), torch.empty(0, dtype=torch.int64, device="cuda"),
                              e.new_empty((0, 8, 64)), e[:, :512], e[:, 512:], None, 0.0, cc, kc, check_status=True)
    assert out.shape == (0, 8, 64)


def test_append_wrapper_checks():
    cc, kc = cache_of(rng_of(4), 1, 16, False)
    kv = torch.zeros((2, 576), dtype=torch.bfloat16, device="cuda")
    q, pos, slots = kv.new_zeros((2, 3, 64)), i32([0, 1]), dev(np.array([0, 1], np.int64))
    ok = dict(positions=pos, slots=slots, q_pe=q, ckv=kv[:, :512], kpe=kv[:, 512:], norm_weight=None, eps=0.0,
              ckv_cache=cc, kpe_cache=kc)
    for bad in (dict(positions=pos.long()), dict(slots=slots.int()), dict(q_pe=q.float()), dict(ckv=kv[:, :500]),
                dict(kpe=kv[:1, 512:]), dict(kpe_cache=kc[:, :8]), dict(positions=pos[:1]), dict(ckv_cache=cc.float()),
                dict(positions=pos.cpu()), dict(norm_weight=kv[0, :512].float()), dict(q_pe_out=q[:, :2])):
        with pytest.raises(ValueError):
            mla.mla_rope_append(mla.rope_spec(FREQ), **{**ok, **bad})
    with pytest.raises(ValueError):
        mla.mla_rope_append(mla.rope_spec(FREQ, [1] * 32), **ok)          # a second axis is wanted
    with pytest.raises(mla.MLAError) as ei:
        mla.mla_rope_append(mla.rope_spec(FREQ), **{**ok, "q_pe": kv.new_zeros((2, 3, 67))[..., 3:]})
    assert ei.value.status == mla.ERR_INVALID_ARG                       # not 16-byte aligned


# ---------------------------------------------------------------------------
# Page summaries
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("P, fp8", [(16, False), (32, True), (64, False), (64, True), (16, True), (32, False)])
def test_summaries_match_oracle(P, fp8):
    rng = rng_of(P, fp8)
    pages, kv_scale = 23, 0.7 if fp8 else 1.0
    cc, kc = cache_of(rng, pages, P, fp8)
    out = torch.full((pages, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    # a prompt's run of slots, single tokens that do or do not complete a page, one page twice, padding
    full = [2, 9, 4, 22, 0]
    slots = [p * P + o for p in full[:3] for o in range(P)] + [22 * P + P - 1, 7 * P + P - 2, -1, 0 * P + P - 1,
                                                             9 * P + P - 1, 5 * P, -P - 1]
    mla.mla_summarize_pages(dev(np.array(slots, np.int64)), cc, kc, out, kv_scale=kv_scale, check_status=True)
    c, k, got = f64(cc.float()) * kv_scale, f64(kc.float()) * kv_scale, f64(out)
    for p in range(pages):
        if p not in full:
            assert np.all(got[p] == 5.0)
            continue
        ref = O.page_mean(c[p], k[p])
        size = np.concatenate([np.abs(c[p]).mean(0), np.abs(k[p]).mean(0)])
        # P additions in fp32, and a product: less than (P + 2) 2^-24 of the mean magnitude
        assert np.all(np.abs(got[p] - ref) <= rounded_bound(ref, False) + size * (P + 2) * 2.0 ** -23), p


@pytest.mark.parametrize("P, fp8", [(16, True), (16, False), (32, True), (64, False)])
def test_summaries_of_a_long_step(P, fp8):
    """Runs of tokens that complete several pages each, an odd number of them too."""
    rng = rng_of(7, P, fp8)
    pages, kv_scale = 40000 // P, 0.25 if fp8 else 1.0
    cc, kc = cache_of(rng, pages, P, fp8)
    out = torch.full((pages, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    slots = (rng.permutation(pages)[:, None] * P + np.arange(P)).astype(np.int64).reshape(-1)
    slots[rng.random(slots.size) < 0.1] = -1                 # padding: some pages are not completed
    mla.mla_summarize_pages(dev(slots), cc, kc, out, kv_scale=kv_scale, check_status=True)
    full = np.zeros(pages, bool)
    full[slots[slots % P == P - 1] // P] = True
    rows = np.concatenate([f64(cc.float()), f64(kc.float())], 2) * kv_scale
    ref, size, got = rows.mean(1), np.abs(rows).mean(1), f64(out)
    assert np.all(got[~full] == 5.0) and 0 < full.sum() < pages
    # as above: P additions in fp32 and a product, and the rounding to bf16
    assert np.all(np.abs(got - ref)[full] <= (rounded_bound(ref, False) + size * (P + 2) * 2.0 ** -23)[full])


def test_summaries_report_a_slot_past_the_cache():
    cc, kc = cache_of(rng_of(5), 2, 16, False)
    out = torch.full((2, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mla.MLAError) as ei:
        mla.mla_summarize_pages(dev(np.array([47], np.int64)), cc, kc, out, check_status=True)
    assert ei.value.status == mla.ERR_DEVICE_BOUNDS and bool((out == 5.0).all())
    mla.mla_summarize_pages(torch.empty(0, dtype=torch.int64, device="cuda"), cc, kc, out, check_status=True)
    with pytest.raises(ValueError):
        mla.mla_summarize_pages(dev(np.array([1], np.int64)), cc, kc, out[:1])


# ---------------------------------------------------------------------------
# Page scores
# ---------------------------------------------------------------------------

def lists_of(rng, counts, num_pages):
    indptr = np.zeros(len(counts) + 1, np.int32)
    indptr[1:] = np.cumsum(counts)
    return indptr, rng.integers(0, num_pages, int(indptr[-1])).astype(np.int32)


@pytest.mark.parametrize("counts, H", [
    ([1], 1), ([5, 0, 130], 16), ([128, 127, 129, 0, 1], 20), ([1000], 128), ([33] * 40, 128), ([300, 2, 77], 7),
    ([0, 0], 16), ([4, 3, 2, 1] * 100, 8), ([513, 64], 40), ([2100], 16), ([700, 701, 1, 699], 100),
    ([300, 1, 5], 49), ([257, 256, 255, 513], 65), ([40, 0, 90], 97), ([129], 127), ([3, 0, 70] * 230, 48),
    ([1, 2, 0, 33, 5] * 200, 56)])
def test_scores_match_oracle(counts, H):
    rng = rng_of(len(counts), sum(counts), H)
    R, num_pages = len(counts), 61
    s = torch.from_numpy(rng.standard_normal((num_pages, 576)).astype(np.float32) * 0.3).to(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((R, H, 576)).astype(np.float32)).to(torch.bfloat16)
    indptr, indices = lists_of(rng, counts, num_pages)
    width = max(counts) + 5
    scores = torch.full((R, width + 3), 9.0, device="cuda")
    mla.mla_page_scores(q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda(), s.cuda(), dev(indptr),
                        dev(indices), scores[:, :width], check_status=True)
    got = f64(scores)
    for r in range(R):
        n = counts[r]
        assert np.all(got[r, n:] == 9.0)
        rows = f64(s)[indices[indptr[r]:indptr[r + 1]]]
        ref = O.page_scores(f64(q[r]), rows) if n else np.zeros(0)
        # 576 exact products accumulated in fp32, in blocks whose sums may be cut rather than rounded:
        # at most 72 steps of 2^-23 of the sum of magnitudes, so less than 2^-16 of it
        size = (np.abs(rows) @ np.abs(f64(q[r])).T).max(1) if n else np.zeros(0)
        assert np.all(np.abs(got[r, :n] - ref) <= size * 2.0 ** -16), r


def test_scores_of_special_values():
    """NaN products lose to any other; a page of which every product is NaN scores -inf; infinities win."""
    q = torch.zeros((1, 2, 576), dtype=torch.bfloat16)
    q[0, 0, 0], q[0, 1, 1] = 1.0, 2.0
    s = torch.zeros((5, 576), dtype=torch.bfloat16)
    s[0, 0] = math.nan                       # NaN for both heads (0 x NaN)
    s[1, 0], s[1, 1] = 3.0, -8.0             # 3, -16
    s[2, 0], s[2, 1] = -3.0, -8.0
    s[3, 0] = math.inf                       # inf for head 0, NaN for head 1
    s[4, 575] = 4.0                          # 0
    scores = torch.zeros((1, 5), device="cuda")
    mla.mla_page_scores(q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda(), s.cuda(), i32([0, 5]),
                        i32([0, 1, 2, 3, 4]), scores, check_status=True)
    assert scores[0].tolist() == [-math.inf, 3.0, -3.0, math.inf, 0.0]


def test_scores_report_bad_lists():
    rng = rng_of(12)
    s = torch.from_numpy(rng.standard_normal((6, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((3, 4, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    qn, qp = q[..., :512].contiguous(), q[..., 512:].contiguous()
    good = torch.zeros((3, 4), device="cuda")
    indices = i32([0, 1, 2, 3, 4, 5])
    mla.mla_page_scores(qn, qp, s, i32([0, 2, 4, 6]), indices, good, check_status=True)

    def bad(indptr, indices, at):
        scores = torch.full((3, 4), 9.0, device="cuda")
        with pytest.raises(mla.MLAError) as ei:
            mla.mla_page_scores(qn, qp, s, i32(indptr), i32(indices), scores, check_status=True)
        assert ei.value.status == mla.ERR_DEVICE_BOUNDS
        for r, c, v in at:
            assert (scores[r, c] == (good[r, c] if v is None else v)), (indptr, r, c)

    bad([0, 2, 4, 6], [0, 6, 2, 3, -1, 5], [(0, 0, None), (0, 1, -math.inf), (1, 1, None), (2, 0, -math.inf), (2, 1, None)])
    bad([0, 2, 4, 7], [0, 1, 2, 3, 4, 5], [(0, 1, None), (1, 0, None), (2, 0, 9.0)])     # past kv_indices
    bad([0, 2, -1, 2], [0, 1, 2, 3, 4, 5], [(0, 0, None), (1, 0, 9.0), (2, 0, 9.0)])     # backwards
    bad([0, 5, 5, 6], [0, 1, 2, 3, 4, 5], [(0, 0, 9.0), (1, 0, 9.0)])                    # longer than a row of scores
    with pytest.raises(ValueError):
        mla.mla_page_scores(qn, qp, s, i32([0, 1]), indices, good)


def test_scores_of_a_list_past_the_columns():
    """Rows of scores further apart than their columns: a list longer than the columns is
    reported by the scores and the selection, and the entries between the rows stay."""
    s = torch.ones((6, 576), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((3, 4, 576), dtype=torch.bfloat16, device="cuda")
    qn, qp, indices = q[..., :512].contiguous(), q[..., 512:].contiguous(), i32([0, 1, 2, 3, 4, 5])
    wide = torch.full((3, 8), 9.0, device="cuda")
    for indptr, written in (([0, 1, 5, 6], (1, 0, 1)), ([0, 1, 2, 6], (1, 1, 0))):
        wide.fill_(9.0)
        with pytest.raises(mla.MLAError) as ei:
            mla.mla_page_scores(qn, qp, s, i32(indptr), indices, wide[:, :3], check_status=True)
        assert ei.value.status == mla.ERR_DEVICE_BOUNDS
        expect = torch.full((3, 8), 9.0)
        for r, n in enumerate(written):
            expect[r, :n] = 576.0
        assert torch.equal(wide.cpu(), expect)
        si, sp = i32([-3] * 4), i32([-3] * 6)
        with pytest.raises(mla.MLAError) as ei:
            mla.mla_select_pages(wide[:, :3], i32(indptr), indices, 2, 0, 1, si, sp, check_status=True)
        assert ei.value.status == mla.ERR_DEVICE_BOUNDS
        assert np.diff(si.cpu()).tolist() == list(written)
        assert sp.tolist() == [indptr[r] for r in range(3) if written[r]] + [-3] * 4


def test_scores_several_tokens_share_a_choice():
    """[R, tokens, heads, .] queries: the best over tokens and heads."""
    rng = rng_of(13)
    s = torch.from_numpy(rng.standard_normal((6, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((2, 3, 16, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    indptr, indices = i32([0, 3, 6]), i32([5, 4, 3, 2, 1, 0])
    qn, qp = q[..., :512].contiguous(), q[..., 512:].contiguous()
    each = torch.zeros((3, 2, 3), device="cuda")
    for j in range(3):
        mla.mla_page_scores(qn[:, j].contiguous(), qp[:, j].contiguous(), s, indptr, indices, each[j])
    both = torch.zeros((2, 3), device="cuda")
    mla.mla_page_scores(qn, qp, s, indptr, indices, both, check_status=True)
    assert torch.allclose(both, each.amax(0), rtol=0, atol=1e-4)


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------

def check_select(scores, counts, k, kf, kl, rng, stride=None):
    R = len(counts)
    indptr, indices = lists_of(rng, counts, 10 ** 6)
    width = max(max(counts), 1)
    wide = torch.full((R, stride or width), math.nan, device="cuda")
    wide[:, :width] = dev(scores.astype(np.float32))[:, :width]
    si = torch.full((R + 1,), -3, dtype=torch.int32, device="cuda")
    sp = torch.full((R * k + 2,), -3, dtype=torch.int32, device="cuda")
    mla.mla_select_pages(wide, dev(indptr), dev(indices), k, kf, kl, si, sp, check_status=True)
    at, got_i, got_p = 0, si.cpu().numpy(), sp.cpu().numpy()
    assert got_i[0] == 0
    for r in range(R):
        ref = O.select_pages(scores[r].astype(np.float32), indices[indptr[r]:indptr[r + 1]], k, kf, kl)
        assert got_i[r + 1] == at + len(ref)
        assert list(got_p[at:at + len(ref)]) == ref, (r, k, kf, kl)
        at += len(ref)
    assert np.all(got_p[at:] == -3)


@pytest.mark.parametrize("counts, k, kf, kl", [
    ([1], 1, 0, 1), ([2, 3, 0, 7], 3, 1, 1), ([31, 32, 33, 1023, 1024, 1025], 32, 1, 2), ([5000, 17, 4999], 256, 4, 4),
    ([200] * 50, 20, 0, 1), ([64, 65], 64, 32, 32), ([9000], 1, 0, 1), ([16384, 20000], 2048, 1, 1), ([70000], 500, 1, 3),
    ([3000, 2999], 2990, 1, 1)])
@pytest.mark.parametrize("kind", ["normal", "few", "equal"])
def test_selection_matches_oracle(counts, k, kf, kl, kind):
    rng = rng_of(sum(counts), k, len(kind))
    shape = (len(counts), max(max(counts), 1))
    s = rng.standard_normal(shape) * 10 if kind == "normal" else \
        rng.integers(-2, 3, shape) * 1.5 if kind == "few" else np.full(shape, -2.5)
    check_select(s, counts, k, kf, kl, rng)


def test_selection_of_special_scores():
    rng = rng_of(21)
    s = rng.standard_normal((4, 300))
    s[0, rng.random(300) < 0.7] = np.nan
    s[1, rng.random(300) < 0.9] = -np.inf
    s[1, rng.random(300) < 0.05] = np.inf
    s[2] = np.where(rng.random(300) < 0.5, 0.0, -0.0)            # equal
    s[3] = np.where(rng.random(300) < 0.5, np.finfo(np.float32).min, -np.inf)
    s[3, ::7] = np.nan
    for k in (2, 40, 150, 299):
        check_select(s, [300, 299, 300, 300], k, 1, 1, rng, stride=333)


def test_selection_reports_bad_lists():
    scores = torch.zeros((3, 4), device="cuda")
    si, sp = i32([-3] * 4), i32([-3] * 6)
    with pytest.raises(mla.MLAError) as ei:
        mla.mla_select_pages(scores, i32([0, 3, 8, 9]), i32(range(9)), 2, 0, 1, si, sp, check_status=True)
    assert ei.value.status == mla.ERR_DEVICE_BOUNDS
    assert si.tolist() == [0, 2, 2, 3] and sp.tolist() == [0, 2, 8, -3, -3, -3]
    mla.mla_select_pages(scores, i32([0, 3, 7, 9]), i32(range(9)), 2, 0, 1, si, sp, check_status=True)
    assert si.tolist() == [0, 2, 4, 6] and sp.tolist() == [0, 2, 3, 6, 7, 8]
    with pytest.raises(mla.MLAError) as ei:
        mla.mla_select_pages(scores, i32([0, 3, 7, 9]), i32(range(9)), 2, 0, 1, si, sp[:5])
    assert ei.value.status == mla.ERR_CAPACITY


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

def speaking(rng, cc, kc, q, pages):
    """Give the rows of `pages` a direction that the query rows share."""
    u = rng.standard_normal(576)
    u /= np.linalg.norm(u)
    q += 6 * u
    for p in pages:
        cc[p] += 10 * u[:512]
        kc[p] += 10 * u[512:]


@pytest.mark.parametrize("lens, H, P, k, q_len, fp8", [
    ([700, 64, 1, 0, 2050], 16, 16, 12, 0, False), ([3000, 5000, 64], 128, 64, 10, 0, False),
    ([900, 33], 16, 32, 8, 4, False), ([2000, 129, 640], 128, 32, 9, 0, True), ([777], 5, 16, 40, 2, False)])
def test_sparse_decoder_matches_oracle(lens, H, P, k, q_len, fp8):
    """Score, select and decode against attention over the pages the oracle selects."""
    rng = rng_of(len(lens), H, k)
    B, Q, kl = len(lens), max(q_len, 1), 2
    counts = [-(-n // P) for n in lens]
    total = sum(counts)
    indptr = np.zeros(B + 1, np.int32)
    indptr[1:] = np.cumsum(counts)
    indices = rng.permutation(total + 2)[:total].astype(np.int32)
    cc, kc = rng.standard_normal((total + 2, P, 512)), rng.standard_normal((total + 2, P, 64))
    q = rng.standard_normal((B, Q, H, 576))
    for b in range(B):
        middle = np.arange(1, max(1, counts[b] - kl))
        rng.shuffle(middle)
        speaking(rng, cc, kc, q[b], indices[indptr[b] + middle[:k - 1 - kl]])
    kv_scale = 0.25 if fp8 else 1.0
    stored = [torch.from_numpy((a / kv_scale).astype(np.float32)).to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
              for a in (cc, kc)]
    cc, kc = (f64(t.float()) * kv_scale for t in stored)
    qb = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    q = f64(qb)
    d_cc, d_kc = (t.cuda() for t in stored)
    # stale rows of pages that are not full are never looked at
    summaries = torch.full((total + 2, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        ends = indices[indptr[b]:indptr[b] + lens[b] // P].astype(np.int64) * P + P - 1
        mla.mla_summarize_pages(dev(ends), d_cc, d_kc, summaries, kv_scale=kv_scale, check_status=True)
    dec = mla.MLASparseDecoder(B * Q, H, max(counts) + 1, k, 1, kl)
    lead = (B, Q, H) if q_len else (B, H)
    sm_scale = 1 / math.sqrt(192.0)
    try:
        dec.plan(indptr, dev(indices), lens, P, sm_scale, q_len=q_len)
        out, lse = dec.run(qb[..., :512].reshape(lead + (512,)).contiguous().cuda(),
                           qb[..., 512:].reshape(lead + (64,)).contiguous().cuda(), d_cc, d_kc, summaries,
                           kv_scale=kv_scale, out_dtype=torch.float32)
        dec.check_status()
        sel, at = dec.sel_indices.cpu().numpy(), dec.sel_indptr.cpu().numpy()
    finally:
        dec.close()
    ref_out, ref_lse = np.zeros((B, Q, H, 512)), np.full((B, Q, H), -np.inf)
    for b in range(B):
        pages = indices[indptr[b]:indptr[b + 1]]
        mean = f64(summaries.float())[pages]
        kept = O.select_pages(O.page_scores(q[b].reshape(-1, 576), mean), pages, k, 1, kl)
        assert list(sel[at[b]:at[b + 1]]) == kept
        if not kept:
            continue
        n = (len(kept) - 1) * P + lens[b] - (counts[b] - 1) * P
        c, r = cc[kept].reshape(-1, 512), kc[kept].reshape(-1, 64)
        for j in range(Q):
            m = n - Q + 1 + j
            s = sm_scale * (q[b, j] @ np.concatenate([c[:m], r[:m]], 1).T)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            ref_lse[b, j] = (top + np.log(p.sum(1, keepdims=True)))[:, 0]
            ref_out[b, j] = p @ c[:m] / p.sum(1, keepdims=True)
    assert_parity(f64(out).reshape(ref_out.shape), f64(lse).reshape(ref_lse.shape), ref_out, ref_lse, "sparse decode")


def test_sparse_decoder_checks():
    with pytest.raises(ValueError):
        mla.MLASparseDecoder(2, 16, 10, 2, 1, 2)
    dec = mla.MLASparseDecoder(2, 16, 4, 3, 1, 1)
    try:
        pages = i32(range(8))
        q = torch.zeros((1, 16, 576), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(mla.MLAError) as ei:
            dec.run(q[..., :512].contiguous(), q[..., 512:].contiguous(), None, None, q)
        assert ei.value.status == mla.ERR_NOT_PLANNED
        with pytest.raises(mla.MLAError) as ei:
            dec.plan([0, 5], pages, [80], 16, 0.1)              # five pages
        assert ei.value.status == mla.ERR_CAPACITY
        with pytest.raises(mla.MLAError):
            dec.plan([0, 1, 2, 3], pages, [1, 1, 1], 16, 0.1)   # three requests
        with pytest.raises(mla.MLAError) as ei:
            dec.plan([0, 2], pages, [32], 16, 0.1, q_len=9)     # 9 x 16 query rows
        assert ei.value.status == mla.ERR_UNSUPPORTED
        for args, kw in ((([0, 2], pages, [33], 16, 0.1), {}), (([0, 3], pages, [33], 16, 0.1), dict(q_len=2)),
                         (([0, 3], pages[:2], [33], 16, 0.1), {}), (([0, 1, 3], pages, [33], 16, 0.1), {})):
            with pytest.raises(ValueError):
                dec.plan(*args, **kw)
    finally:
        dec.close()


def test_sparse_decoder_refuses_another_head_count():
    """The decode would read the planned heads of every request, past the queries."""
    dec = mla.MLASparseDecoder(2, 16, 4, 3, 1, 2)
    try:
        cache = torch.zeros((8, 16, 576), dtype=torch.bfloat16, device="cuda")
        cache = cache[..., :512].contiguous(), cache[..., 512:].contiguous()
        s = torch.zeros((8, 576), dtype=torch.bfloat16, device="cuda")
        for q_len, shapes in ((0, [(1, 8), (1, 32), (1, 2, 16)]), (2, [(1, 16), (1, 1, 16), (1, 2, 8)])):
            dec.plan([0, 2], i32(range(2)), [20], 16, 0.1, q_len=q_len)
            for lead in shapes:
                q = torch.zeros(lead + (576,), dtype=torch.bfloat16, device="cuda")
                with pytest.raises(ValueError):
                    dec.run(q[..., :512].contiguous(), q[..., 512:].contiguous(), *cache, s)
    finally:
        dec.close()


def test_calls_on_another_stream():
    """Every operator queued on a stream that is not the current one, while the current one is held up."""
    side = torch.cuda.Stream()
    rng = rng_of(41)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    q, kv, pos, slots = bf(9, 16, 64), bf(9, 576), i32(range(9)), dev(np.arange(7, 16))
    cc, kc = cache_of(rng, 2, 16, False)
    summaries = torch.full((2, 576), math.nan, dtype=torch.bfloat16, device="cuda")
    scores = torch.full((1, 2), math.nan, device="cuda")
    si, sp, indptr, indices = i32([-1, -1]), i32([-1, -1]), i32([0, 2]), i32([1, 0])
    qn = bf(1, 16, 512)
    s = tables_state(rng, [5], 16, 4, spare=2)
    t = [i32(s["lens"]), i32([3]), dev(s["table"]), dev(s["free"]), i32([2])]
    o = [i32([-1] * 2), i32([-1] * 4), i32([-1] * 2), dev(np.full(4, -9)), i32([-1] * 4), i32([-1])]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                        # about 0.1 s on the current stream
    out = mla.mla_rope_append(mla.rope_spec(FREQ), pos, slots, q, kv[:, :512], kv[:, 512:], None, 0.0, cc, kc,
                              torch.empty_like(q), stream=side)
    mla.mla_summarize_pages(slots, cc, kc, summaries, stream=side)
    mla.mla_summarize_pages(dev_on(side, np.array([31])), cc, kc, summaries, stream=side)
    mla.mla_page_scores(qn, q[:1], summaries, indptr, indices, scores, stream=side)
    mla.mla_select_pages(scores, indptr, indices, 1, 0, 1, si, sp, stream=side)
    mla.mla_build_tables(*t[:2], *t[2:5], 16, *o[:5], o[5], stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        assert not summaries.isnan().any() and not scores.isnan().any()
        assert si.tolist() == [0, 1] and sp.tolist() == [0, -1] and o[5].tolist() == [0] and t[0].tolist() == [8]
        ref = O.page_mean(f64(cc[0]), f64(kc[0]))
        assert np.abs(f64(summaries[0]) - ref).max() < 0.05
    torch.cuda.synchronize()


def dev_on(stream, a):
    with torch.cuda.stream(stream):
        return dev(a)


def test_outputs_made_on_another_stream():
    """An output that a call makes for another stream is not memory that the current
    stream gave back and has yet to read."""
    side = torch.cuda.Stream()
    T, H, B = 1024, 128, 128    # outputs of 16 MB, blocks of their own
    q_pe = torch.zeros((T, H, 64), dtype=torch.bfloat16, device="cuda")
    ckv, kpe = (torch.zeros((T, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64))
    cache = [torch.zeros((8, 16, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64)]
    pos, slots = i32(np.zeros(T)), torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[:32] = torch.arange(32, device="cuda")
    qn, qp = (torch.zeros((B, H, n), dtype=torch.bfloat16, device="cuda") for n in (512, 64))
    s = torch.zeros((8, 576), dtype=torch.bfloat16, device="cuda")
    dec = mla.MLASparseDecoder(B, H, 2, 2)
    dec.plan(range(B + 1), i32(np.arange(B) % 8), [16] * B, 16, 0.1)
    torch.cuda.synchronize()

    def behind(shape, call):
        call()                               # (loads its kernels)
        before = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
        copy = torch.empty_like(before)
        torch.cuda.synchronize()
        torch.cuda._sleep(1 << 27)           # the current stream is busy for some tens of milliseconds
        copy.copy_(before)                   # and reads its tensor after that
        del before
        made = call()                        # meanwhile another stream has an output of the same size
        torch.cuda.synchronize()
        assert bool((copy == 1).all())
        return made

    try:
        spec = mla.rope_spec(FREQ)
        turned = behind((T, H, 64), lambda: mla.mla_rope_append(spec, pos, slots, q_pe, ckv, kpe, None, 0.0, *cache,
                                                                 stream=side))
        assert bool((turned[:32] == 0).all())
        out, lse = behind((B, H, 512), lambda: dec.run(qn, qp, *cache, s, stream=side))
        assert bool((out == 0).all())
    finally:
        dec.close()


def test_offsets_past_32_bits():
    """The last slot of a cache of more than 2^31 values, and the last of more than 2^31 summary values."""
    pages, P = 66000, 64
    cc = torch.zeros((pages, P, 512), dtype=torch.float8_e4m3fn, device="cuda")
    kc = torch.zeros((pages, P, 64), dtype=torch.float8_e4m3fn, device="cuda")
    assert cc.numel() > 2 ** 31
    kv = torch.full((1, 576), 2.0, dtype=torch.bfloat16, device="cuda")
    slot = dev(np.array([pages * P - 1], np.int64))
    mla.mla_rope_append(mla.rope_spec(FREQ), i32([0]), slot, None, kv[:, :512], kv[:, 512:], None, 0.0, cc, kc,
                        check_status=True)
    assert bool((cc[-1, -1].float() == 2).all()) and bool((kc[-1, -1].float() == 2).all())
    assert int(cc.view(torch.int64).count_nonzero()) == 64      # nothing else was written
    summaries = torch.empty((pages, 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_summarize_pages(slot, cc, kc, summaries, check_status=True)
    assert bool((summaries[-1] == 2 / 64).all())
    del cc, kc
    many = 2 ** 31 // 576 + 5
    summaries = torch.empty((many, 576), dtype=torch.bfloat16, device="cuda")
    summaries[-1], summaries[0] = 3.0, 1.0
    for H in (16, 128):
        q = torch.ones((1, H, 576), dtype=torch.bfloat16, device="cuda")
        scores = torch.zeros((1, 2), device="cuda")
        mla.mla_page_scores(q[..., :512].contiguous(), q[..., 512:].contiguous(), summaries, i32([0, 2]),
                            i32([many - 1, 0]), scores, check_status=True)
        assert scores.tolist() == [[3 * 576.0, 576.0]]
    # a page table whose rows lie 2^30 entries apart
    wide = torch.full((3 * 2 ** 30,), -1, dtype=torch.int32, device="cuda")
    table = wide.view(3, 2 ** 30)[:, :4]
    o = [i32([-1] * 4), i32([-1] * 12), i32([-1] * 4), dev(np.full(18, -9)), i32([-1] * 18), i32([-1])]
    mla.mla_build_tables(i32([0, 0, 0]), i32([1, 0, 17]), table, i32([5, 4, 3, 2, 1, 0]), i32([6]), 16, *o)
    assert o[5].tolist() == [0] and o[0].tolist() == [0, 1, 1, 3] and o[1].tolist()[:3] == [0, 1, 2]
    assert table[2].tolist() == [1, 2, -1, -1] and table[0].tolist() == [0, -1, -1, -1]


def test_calls_at_once_on_several_threads():
    """Calls of different sizes at the same time from several host threads, each on its own stream: the results of
    the calls one by one."""
    import threading
    rng = rng_of(61)
    s = torch.from_numpy(rng.standard_normal((900, 576)).astype(np.float32) * 0.3).to(torch.bfloat16).cuda()
    jobs = []
    for counts, H, k in (([90, 3], 16, 8), ([3] * 600, 128, 2), ([400], 128, 64), ([12000, 9000], 40, 100)):
        q = torch.from_numpy(rng.standard_normal((len(counts), H, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
        indptr, indices = lists_of(rng, counts, 900)
        jobs.append(dict(qn=q[..., :512].contiguous(), qp=q[..., 512:].contiguous(), indptr=dev(indptr),
                         indices=dev(indices), k=k, n=len(counts), w=max(counts)))

    def call(j, stream):
        scores = torch.zeros((j["n"], j["w"]), device="cuda")
        si, sp = i32([0] * (j["n"] + 1)), i32([0] * (j["n"] * j["k"]))
        torch.cuda.synchronize()
        for _ in range(60):
            mla.mla_page_scores(j["qn"], j["qp"], s, j["indptr"], j["indices"], scores, stream=stream)
            mla.mla_select_pages(scores, j["indptr"], j["indices"], j["k"], 0, 1, si, sp, stream=stream)
        return scores, si, sp

    streams = [torch.cuda.Stream() for _ in jobs]
    alone = [call(j, st) for j, st in zip(jobs, streams)]
    torch.cuda.synchronize()
    got, failed = [None] * len(jobs), []

    def work(i):
        try:
            got[i] = call(jobs[i], streams[i])
        except Exception as e:                                # a refused launch, say
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_sparse_decoder_replays_smaller_plans():
    """A run captured for three requests replays a later plan of two, and the three again."""
    rng = rng_of(51)
    B, H, P, W = 3, 16, 16, 40
    lens = [300, 17, 620]
    cc, kc = cache_of(rng, B * W, P, False)
    summaries = torch.cat([cc.float().mean(1), kc.float().mean(1)], 1).to(torch.bfloat16)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    qn, qp = bf(B, H, 512), bf(B, H, 64)
    pages = i32(rng.permutation(B * W))
    out = torch.zeros((B, H, 512), device="cuda")
    lse = torch.zeros((B, H), device="cuda")
    dec, ref = mla.MLASparseDecoder(B, H, W, 9, 1, 1), mla.MLASparseDecoder(B, H, W, 9, 1, 1)

    def indptr_of(n):
        return np.concatenate([[0], np.cumsum([-(-x // P) for x in n])]).astype(np.int32)

    def expect(n, k):
        ref.plan(indptr_of(n), pages, n, P, 0.07)
        return ref.run(qn[:k].contiguous(), qp[:k].contiguous(), cc, kc, summaries, out_dtype=torch.float32)

    try:
        dec.plan(indptr_of(lens), pages, lens, P, 0.07)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dec.run(qn, qp, cc, kc, summaries, out, lse)
        for n in (lens, [639, 5], [16, 640], [0], lens):
            dec.plan(indptr_of(n), pages, n, P, 0.07)
            out.fill_(math.nan)
            g.replay()
            o, l = expect(n, len(n))
            assert torch.equal(out[:len(n)], o) and torch.equal(lse[:len(n)], l)
            assert bool(out[len(n):].isnan().all())              # rows past the batch stay as they were
        with pytest.raises(mla.MLAError):
            dec.plan([0], pages, [], P, 0.07)                    # a batch of none, as for MLADecoder
        dec.check_status()
    finally:
        dec.close()
        ref.close()


def test_steps_together_from_a_graph():
    """Serving steps -- tables, append, summaries, choice, decode -- captured once and replayed, against a model of
    the requests' tokens in numpy; the same steps eagerly on another stream give the same bits."""
    B, H, P, W, k, steps = 3, 16, 16, 24, 6, 20
    rng = rng_of(77)
    lens0 = [100, 15, 230]
    s = tables_state(rng, [0] * B, P, W, spare=B * W)
    freq_rope = mla.rope_spec(FREQ)
    sm_scale = 1 / math.sqrt(192.0)
    bf = lambda *sh: torch.from_numpy(rng.standard_normal(sh).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    prompt_kv, step_kv, step_q = bf(sum(lens0), 576), bf(steps, B, 576), bf(steps, B, H, 576)
    weight = bf(512)

    def serve(graphed, stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            kv_len, table, free, count = i32([0] * B), dev(s["table"]), dev(s["free"]), i32([s["count"]])
            o = {n: torch.zeros(z, dtype=torch.int32, device="cuda") for n, z in
                 dict(indptr=B + 1, indices=B * W, q=B + 1, pos=sum(lens0), status=1).items()}
            slots = torch.zeros(sum(lens0), dtype=torch.int64, device="cuda")
            cc = torch.full((s["count"], P, 512), math.nan, dtype=torch.bfloat16, device="cuda")
            kc = torch.full((s["count"], P, 64), math.nan, dtype=torch.bfloat16, device="cuda")
            summaries = torch.full((s["count"], 576), math.nan, dtype=torch.bfloat16, device="cuda")
            new = i32(lens0)
            kv, q = prompt_kv.clone(), step_q[0].clone()
            qr = torch.zeros((B, H, 64), dtype=torch.bfloat16, device="cuda")
            out = torch.zeros((B, H, 512), dtype=torch.float32, device="cuda")
            lse = torch.zeros((B, H), dtype=torch.float32, device="cuda")
            dec = mla.MLASparseDecoder(B, H, W, k, 1, 2)

            def tables(n):
                mla.mla_build_tables(kv_len, new, table, free, count, P, o["indptr"], o["indices"], o["q"], slots[:n],
                                     o["pos"][:n], o["status"])

            def append(n, queries):
                mla.mla_rope_append(freq_rope, o["pos"][:n], slots[:n], queries, kv[:n, :512], kv[:n, 512:], weight,
                                    1e-6, cc, kc, q_pe_out=None if queries is None else qr)
                mla.mla_summarize_pages(slots[:n], cc, kc, summaries)

            def step():
                tables(B)
                append(B, q[..., 512:])
                dec.run(qn, qr, cc, kc, summaries, out, lse)

            tables(sum(lens0))
            append(sum(lens0), None)
            new.fill_(1)
            lens = list(lens0)
            results, g = [], None
            qn = torch.zeros((B, H, 512), dtype=torch.bfloat16, device="cuda")
            for i in range(steps):
                lens = [n + 1 for n in lens]
                indptr = np.concatenate([[0], np.cumsum([-(-n // P) for n in lens])]).astype(np.int32)
                kv[:B].copy_(step_kv[i])
                q.copy_(step_q[i])
                qn.copy_(q[..., :512])
                dec.plan(indptr, o["indices"], lens, P, sm_scale, stream=stream)
                if graphed and g is None:
                    stream.synchronize()
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=stream):
                        step()
                if graphed:
                    g.replay()
                else:
                    step()
                assert int(o["status"]) == 0
                results.append((out.clone(), lse.clone(), dec.sel_indices[:int(dec.sel_indptr[-1])].clone()))
            dec.check_status()
            stream.synchronize()
            state = f64(cc), f64(kc), f64(summaries), table.cpu().numpy(), kv_len.cpu().numpy()
            dec.close()
            return results, state

    got, state = serve(True, torch.cuda.Stream())
    again, _ = serve(False, torch.cuda.Stream())
    for a, b in zip(got, again):
        assert all(torch.equal(x, y) for x, y in zip(a, b))

    cc, kc, summaries, table, kv_len = state
    assert list(kv_len) == [n + steps for n in lens0]
    # the cache holds every token where the table says, in order
    for b in range(B):
        first = int(sum(lens0[:b]))
        rows = np.concatenate([f64(prompt_kv[first:first + lens0[b]]), f64(step_kv[:, b])])
        n = len(rows)
        pages = table[b, :-(-n // P)]
        c, r = cc[pages].reshape(-1, 512)[:n], kc[pages].reshape(-1, 64)[:n]
        ref = O.norm_row(rows[:, :512], f64(weight), 1e-6)
        assert np.all(np.abs(c - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -18))
        for t in range(n):
            ref = O.rotate(rows[t, 512:], [t], FREQ, [0] * 32, False)
            assert np.all(np.abs(r[t] - ref) <= np.abs(ref) * 2.0 ** -8 + np.abs(rows[t, 512:]).max() * 2.0 ** -19)
        # and the last step's decode is attention over the pages it chose
        out, lse, sel = got[-1]
        kept_n = [min(k, -(-int(x) // P)) for x in kv_len]
        kept = sel.cpu().numpy()[sum(kept_n[:b]):sum(kept_n[:b + 1])]
        where = [list(pages).index(p) for p in kept]
        assert where == sorted(where) and where[0] == 0 and where[-2:] == [len(pages) - 2, len(pages) - 1]
        qq = f64(step_q[steps - 1, b])
        q_rot = O.rotate(qq[:, 512:], [n - 1], FREQ, [0] * 32, False)
        q_rot = f64(torch.from_numpy(q_rot.astype(np.float32)).to(torch.bfloat16))
        m = (len(kept) - 1) * P + n - (len(pages) - 1) * P
        cs, rs = cc[kept].reshape(-1, 512)[:m], kc[kept].reshape(-1, 64)[:m]
        sc = sm_scale * (qq[:, :512] @ cs.T + q_rot @ rs.T)
        p = np.exp(sc - sc.max(1, keepdims=True))
        assert_parity(f64(out[b]), f64(lse[b]), p @ cs / p.sum(1, keepdims=True),
                      sc.max(1) + np.log(p.sum(1)), "last step")
        # the chosen middle pages score no lower than the others, but for what fp32 may turn around
        qf = np.concatenate([qq[:, :512], q_rot], 1)
        score = O.page_scores(qf, summaries[pages])
        others = [i for i in range(1, len(pages) - 2) if i not in where]
        middle = [i for i in where if 1 <= i < len(pages) - 2]
        if others and middle:
            assert score[middle].min() >= score[others].max() - 1e-2
