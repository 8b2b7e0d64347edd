"""lora_rms_norm against the formula in 64 bits.

Tolerances: y is one bf16 rounding (2^-8 of the value) of an fp32 result
whose sum of squares is at most 2^-17 off (at most 64 terms are added in a
row, then pairwise); a scale is that result's maximum; a code is one e4m3
rounding: 2^-4 of the value, or half the smallest step, 2^-10, times the scale.
"""
import numpy as np
import pytest
import torch

import kv4_ref as R
from lora_serving_gb300 import abi, build

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _inputs(T, W, seed, res=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (r(T, W).bfloat16(), (3 * r(T, W)).bfloat16() if res else None, (1 + 0.3 * r(W)).bfloat16())


def _check(T, W, group, x, res, w, eps, y, h, y8, sc):
    hr, n = R.norm(R.f64(x), R.f64(w), eps, None if res is None else R.f64(res))
    if res is not None:
        assert np.array_equal(R.f64(h), hr)
    if y is not None:
        assert (np.abs(R.f64(y) - n) <= (2.0 ** -8 + FP32) * np.abs(n) + 1e-38).all()
    if y8 is not None:
        size = group or W
        for i in range(-(-W // size)):
            part = n[:, i * size:(i + 1) * size]
            s = np.abs(part).max(1) / 448
            got = R.f64(sc)[:, i]
            assert (np.abs(got - s) <= FP32 * s).all()
            val = R.f64(y8[:, i * size:(i + 1) * size].float()) * got[:, None]
            assert (np.abs(val - part) <= (2.0 ** -4 + 2 * FP32) * np.abs(part) + 2.0 ** -10 * s[:, None]).all()


@pytest.mark.parametrize("T,W", [(1, 8), (3, 72), (5, 128), (2, 136), (64, 1000), (7, 4096), (3, 4104), (2, 8192),
                                 (1, 14336), (2, 32776), (1, 65536), (1021, 2568)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm(T, W, group):
    x, res, w = _inputs(T, W, T * 7 + W)
    y, h = torch.empty_like(x), torch.empty_like(x)
    y8 = torch.empty(T, W, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(T, -(-W // group) if group else 1, device="cuda")
    abi.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=h, y=y, y8=y8, scales=sc, group=group)
    _check(T, W, group, x, res, w, 1e-5, y, h, y8, sc)


@pytest.mark.parametrize("what", ["y", "y8"])
def test_norm_one_output_no_residual(what):
    x, _, w = _inputs(33, 520, 5, res=False)
    y = torch.empty_like(x) if what == "y" else None
    y8 = torch.empty(33, 520, dtype=torch.float8_e4m3fn, device="cuda") if what == "y8" else None
    sc = torch.empty(33, 5, device="cuda") if what == "y8" else None
    abi.lora_rms_norm(x, w, 0.0, y=y, y8=y8, scales=sc, group=128)
    _check(33, 520, 128, x, None, w, 0.0, y, None, y8, sc)


def test_norm_strided_rows_and_in_place():
    T, W = 37, 264
    x, res, w = _inputs(T, W + 40, 11)
    wide = [t[:, 16:16 + W] for t in (x, res)]
    keep = [t.clone() for t in wide]
    sc = torch.full((T, 6), -1.0, device="cuda")
    y8 = torch.zeros(T, W + 8, dtype=torch.float8_e4m3fn, device="cuda")
    # h over the residual, y over x
    abi.lora_rms_norm(wide[0], w[:W].contiguous(), 1e-6, residual=wide[1], residual_out=wide[1], y=wide[0],
                      y8=y8[:, :W], scales=sc, group=128)
    _check(T, W, 128, keep[0], keep[1], w[:W], 1e-6, wide[0], wide[1], y8[:, :W], sc[:, :3])
    assert (sc[:, 3:] == -1).all()                                 # nothing outside the groups
    assert (y8[:, W:].float() == 0).all()
    fresh = _inputs(T, W + 40, 11)
    assert torch.equal(x[:, :16], fresh[0][:, :16]) and torch.equal(res[:, 16 + W:], fresh[1][:, 16 + W:])


def test_norm_zero_and_nan_rows():
    x, res, w = _inputs(4, 256, 3)
    x[1], res[1] = 0, 0
    x[2, 7] = float("nan")
    x[3, :128] = 0
    res[3, :128] = 0                                               # one group of zeros
    y, h = torch.empty_like(x), torch.empty_like(x)
    y8 = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 2, device="cuda")
    abi.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=h, y=y, y8=y8, scales=sc, group=128)
    assert (y[1] == 0).all() and (sc[1] == 0).all() and (y8[1].float() == 0).all()
    assert y[2].isnan().all() and sc[2].isnan().all() and y8[2].float().isnan().all()
    assert sc[3, 0] == 0 and (y8[3, :128].float() == 0).all() and sc[3, 1] > 0
    keep = [0, 3]
    hr, n = R.norm(R.f64(x[keep]), R.f64(w), 1e-5, R.f64(res[keep]))
    assert (np.abs(R.f64(y[keep]) - n) <= (2.0 ** -8 + FP32) * np.abs(n)).all()


def test_norm_on_its_own_stream_and_empty():
    x, res, w = _inputs(256, 4096, 9)
    h, y = torch.empty_like(x), torch.empty_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    abi.lora_rms_norm(x, w, 1e-5, residual=res, residual_out=h, y=y, stream=st)
    st.synchronize()
    _check(256, 4096, 0, x, res, w, 1e-5, y, h, None, None)
    abi.lora_rms_norm(x[:0], w, 1e-5, y=y[:0])
