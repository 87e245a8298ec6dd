"""The 4-bit decode's partition, compiled from the planner's C++ alone (no GPU)."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <algorithm>
#include "planner.h"
using namespace mla;
extern "C" int partition(const int32_t* indptr, const int32_t* len, int batch, int workers, int rows, int32_t* units,
                         int32_t* worker_ptr, int32_t* merge, int32_t* counts, double* us) {
  Partition p, even;
  partition_batch_q4(indptr, len, batch, workers, rows, &p);
  partition_batch(indptr, len, batch, workers, kTileTc, q4_costs(rows), &even);
  us[0] = q4_step_estimate_us(p, rows);
  us[1] = q4_step_estimate_us(even, rows);
  for (size_t i = 0; i < p.units.size(); ++i) {
    const WorkUnit& u = p.units[i];
    const int32_t v[] = {u.req, u.tok_begin, u.tok_end, u.out_slot, u.page_base, u.kv_len};
    std::copy(v, v + 6, units + 6 * i);
  }
  std::copy(p.worker_ptr.begin(), p.worker_ptr.end(), worker_ptr);
  for (size_t i = 0; i < p.merge.size(); ++i) {
    const int32_t v[] = {p.merge[i].req, p.merge[i].first_slot, p.merge[i].n_slots};
    std::copy(v, v + 3, merge + 3 * i);
  }
  counts[0] = static_cast<int32_t>(p.units.size());
  counts[1] = p.n_slots;
  counts[2] = static_cast<int32_t>(p.merge.size());
  return 0;
}
"""


@pytest.fixture(scope="module")
def partition(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("planner")
    (d / "harness.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "paged_mla_decode_02_gb300", "csrc")
    out = str(d / "planner.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", csrc, "-I", os.path.join(ROOT, "include"),
                    str(d / "harness.cpp"), os.path.join(csrc, "planner.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    P = lambda a: a.ctypes.data_as(ctypes.c_void_p)

    def call(lens, rows, workers, page=64):
        lens = np.array(lens, np.int32)
        indptr = np.concatenate([[0], np.cumsum(-(-lens // page))]).astype(np.int32)
        units, ptr = np.zeros((workers + len(lens), 6), np.int32), np.full(workers + 1, -1, np.int32)
        merge, counts, us = np.zeros((len(lens), 3), np.int32), np.zeros(3, np.int32), np.zeros(2)
        lib.partition(P(indptr), P(lens), len(lens), workers, rows, P(units), P(ptr), P(merge), P(counts), P(us))
        return indptr, units[:counts[0]], ptr, merge[:counts[2]], int(counts[1]), us
    return call


@pytest.mark.parametrize("seed, batch, longest, rows", [
    (1, 1, 200000, 16), (2, 4, 2000, 16), (3, 64, 4096, 128), (4, 128, 8192, 128), (5, 700, 200, 24), (6, 3, 5, 64), (7, 33, 70000, 32),
    (8, 4096, 300, 16)])
def test_every_token_is_in_one_unit(partition, seed, batch, longest, rows):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, batch)
    lens[0] = longest
    workers = 152 // -(-rows // 64)
    indptr, units, ptr, merge, n_slots, us = partition(lens, rows, workers)
    assert len(units) <= workers + batch and n_slots <= workers + batch
    # what a plan's buffers of shares hold: a row for every worker and 128 query rows, and the requests' own
    assert n_slots * rows <= 152 * 128 + batch * rows
    assert ptr[0] == 0 and ptr[-1] == len(units) and (np.diff(ptr) >= 0).all()
    seen = np.zeros(batch, np.int64)
    for req, begin, end, slot, base, n in units:
        assert begin == seen[req] and begin % 128 == 0 and begin < end <= lens[req] and n == lens[req] and base == indptr[req]
        assert end == lens[req] or end % 128 == 0
        seen[req] = end
    np.testing.assert_array_equal(seen, lens)
    # shares: the units of a cut request take the slots of its entry in their order
    merged = {int(r): (int(s), int(k)) for r, s, k in merge}
    taken = 0
    for req in range(batch):
        mine = units[units[:, 0] == req]
        if len(mine) == 1:
            assert mine[0, 3] == -1 and req not in merged
        elif len(mine) == 0:
            assert lens[req] == 0 and merged[req][1] == 0
        else:
            assert merged[req][1] == len(mine) and list(mine[:, 3]) == list(range(merged[req][0], merged[req][0] + len(mine)))
            taken += len(mine)
    assert taken == n_slots
    assert us[0] <= us[1]                      # never a partition that is estimated worse than the even one


def test_short_requests_are_cut_and_even_ones_left_whole(partition):
    _, units, _, _, n_slots, _ = partition([2000, 1500, 700, 300], 16, 152)
    assert n_slots == len(units) == sum(-(-n // 128) for n in (2000, 1500, 700, 300))      # single tiles
    _, units, _, _, n_slots, _ = partition([4096] * 64, 128, 76)
    assert len(units) == 64 and n_slots == 0
    _, units, ptr, _, n_slots, _ = partition([131072] * 4, 16, 152)
    assert n_slots == len(units) == 152 and (np.diff(ptr) == 1).all()
