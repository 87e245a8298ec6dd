"""Rows read back out of a paged cache: what test_gpu_q4.py leaves out."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_mla_decode_02_gb300 import mla
from test_gpu_q4 import i32, rng_of

TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


def round_once(x, dtype):
    """float64 numbers to the nearest of the type, ties to even, as float64."""
    bits, least, top = dict(bf16=(8, -133, 2.0 ** 128), fp16=(11, -24, 2.0 ** 16), fp32=(24, -149, 2.0 ** 128))[dtype]
    _, e = np.frexp(x)                                        # |x| in [2^(e - 1), 2^e)
    unit = np.exp2(np.maximum(e - bits, least).astype(float))
    y = np.rint(x / unit) * unit
    return np.where(np.abs(y) >= top, np.copysign(np.inf, y), y)


def codes():
    """The 254 e4m3 numbers as float64, and their codes."""
    c = np.array([i for i in range(256) if i & 127 != 127], np.uint8)
    return torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy(), c


def twice_rounded_scales(rng, dtype, power):
    """Scales near 2^power under which some e4m3 number's product, rounded to fp32 and
    then to the type, is not the product rounded once."""
    values, _ = codes()
    found = []
    while len(found) < 3:
        s = (1 + rng.random(20000)).astype(np.float32) * np.float32(2.0 ** power)
        exact = values[None, 8:16] * s[:, None].astype(np.float64)     # a number for each of the eight significands
        wrong = round_once(exact, dtype) != round_once(round_once(exact, "fp32"), dtype)
        found += list(s[wrong.any(1)])
    return [float(x) for x in found[:3]]


def test_round_once_on_the_cpu():
    x = np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, -1 - 2.0 ** -9, 2.0 ** -133, 2.0 ** -135, 0.0, 3e38])
    want = [1, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -1, 2.0 ** -133, 0, 0, float(torch.tensor(3e38).bfloat16())]
    np.testing.assert_array_equal(round_once(x, "bf16"), want)
    x = np.float32(rng_of(90).standard_normal(1000)).astype(np.float64)
    for dtype in ("bf16", "fp16"):
        np.testing.assert_array_equal(round_once(x, dtype), torch.from_numpy(x).float().to(TYPES[dtype]).double().numpy())
    assert all(s > 0 for s in twice_rounded_scales(rng_of(91), "fp16", -3))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("power", [-3, 0, 5, -12, -128, 119])
def test_e4m3_rows_under_scales_of_all_bits(dtype, power):
    """kv_scale is not a power of two: every code of both signs, rounded once."""
    values, c = codes()
    rng = rng_of(92, power + 200)
    P, n = 16, 16
    flat = np.resize(rng.permutation(np.tile(c, 40)), n * 576).reshape(n, 576)
    flat[0, :254] = c
    cache = torch.from_numpy(flat).cuda().view(torch.float8_e4m3fn)
    ckv, kpe = cache[:, :512].contiguous().view(1, P, 512), cache[:, 512:].contiguous().view(1, P, 64)
    stood = torch.from_numpy(flat).view(torch.float8_e4m3fn).double().numpy()
    scales = [0.1, 1 / 3, 0.7] if power == 0 else [float(np.float32(2.0 ** power * f)) for f in (1.1, 1.7)]
    if dtype != "fp32" and power in (-3, 0, 5):
        scales += twice_rounded_scales(rng, dtype, power)
    for scale in scales:
        out, pe = torch.zeros(n, 512, dtype=TYPES[dtype], device="cuda"), torch.zeros(n, 64, dtype=TYPES[dtype], device="cuda")
        mla.mla_read_cache(ckv, kpe, i32([0, 1]), i32([0]), i32([0]), i32([0, n]), out, pe, kv_scale=scale, check_status=True)
        got = torch.cat([out, pe], 1).double().cpu().numpy()
        want = round_once(stood * float(np.float32(scale)), dtype)
        np.testing.assert_array_equal(got, want, err_msg=str(scale))
        np.testing.assert_array_equal(np.signbit(got), np.signbit(stood))


@pytest.mark.gpu
def test_e4m3_nan_stays():
    flat = np.full((16, 576), 0x7f, np.uint8)
    flat[:, ::2] = 0xff
    cache = torch.from_numpy(flat).cuda().view(torch.float8_e4m3fn)
    for dtype in TYPES.values():
        out, pe = torch.zeros(16, 512, dtype=dtype, device="cuda"), torch.zeros(16, 64, dtype=dtype, device="cuda")
        mla.mla_read_cache(cache[:, :512].contiguous().view(1, 16, 512), cache[:, 512:].contiguous().view(1, 16, 64),
                           i32([0, 1]), i32([0]), i32([0]), i32([0, 16]), out, pe, kv_scale=0.3, check_status=True)
        assert out.isnan().all() and pe.isnan().all()


@pytest.mark.gpu
def test_rows_past_outputs_of_no_rows_are_reported():
    cache = torch.zeros(2, 16, 304, dtype=torch.uint8, device="cuda")
    ckv, pe = torch.zeros(0, 512, device="cuda"), torch.zeros(0, 64, device="cuda")
    with pytest.raises(mla.MLAError) as e:
        mla.mla_read_cache(cache, None, i32([0, 1]), i32([0]), i32([0]), i32([0, 3]), ckv, pe, check_status=True)
    assert e.value.status == mla.ERR_DEVICE_BOUNDS
    mla.mla_read_cache(cache, None, i32([0, 1]), i32([0]), i32([0]), i32([0, 0]), ckv, pe, check_status=True)
    mla.mla_read_cache(cache, None, i32([0]), i32([]), i32([]), i32([0]), ckv, pe, check_status=True)
