"""The 8-bit output of lora_rms_norm where a group's largest value is far below
fp32's normal range times 448: 448 / max |n| is then no fp32 number.

Tolerances as in test_gpu_rms_norm.py, and in addition what a scale loses
when it is one of fp32's subnormal numbers: 2^-150, and 448 times that for the
value that a code stands for.  Products of three factors round to subnormal
numbers twice: another 2^-149 of n."""
import numpy as np
import pytest
import torch

import kv4_ref as R
from lora_serving_gb300 import abi, build

pytestmark = pytest.mark.gpu
FP32, TINY = 2.0 ** -17, 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("values", [[1e-37], [1e-38], [-1e-36, 3e-37, 1e-37, 2e-39], [1e-39, 1e-40], [-1e-34], [1e-30, 1e-37], [2e-40]])
def test_small_values_beside_zeros(values, group):
    W = 512
    x = torch.zeros(3, W)
    if group:   # other groups as usual: the row's rms is about 1
        x[:, 128:384] = torch.randn(3, 256, generator=torch.Generator().manual_seed(1))
    x[0, 3:3 + 40 * len(values):40] = torch.tensor(values)
    x[1, 511 - len(values) + 1:] = torch.tensor(values)
    x[2, :64] = torch.tensor(values).repeat(64)[:64]
    x = x.bfloat16().cuda()
    w = (1 + 0.3 * torch.randn(W, generator=torch.Generator().manual_seed(2))).bfloat16().cuda()
    y, y8 = torch.empty_like(x), torch.empty(3, W, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(3, 4 if group else 1, device="cuda")
    abi.lora_rms_norm(x, w, 1e-5, y=y, y8=y8, scales=sc, group=group)
    _, n = R.norm(R.f64(x), R.f64(w), 1e-5)
    codes, size = R.f64(y8.float()), group or W
    assert np.isfinite(codes).all() and np.isfinite(R.f64(sc)).all()
    for i in range(W // size):
        part, got = n[:, i * size:(i + 1) * size], R.f64(sc)[:, i]
        s = np.abs(part).max(1) / 448
        assert (np.abs(got - s) <= FP32 * s + 2 * TINY).all()
        val = codes[:, i * size:(i + 1) * size] * got[:, None]
        assert (np.abs(val - part) <= (2.0 ** -4 + 2 * FP32) * np.abs(part) + 2.0 ** -10 * s[:, None] + 2 * 448 * TINY).all()
        zero = part == 0
        assert (codes[:, i * size:(i + 1) * size][zero] == 0).all()
    assert (np.abs(R.f64(y) - n) <= (2.0 ** -8 + FP32) * np.abs(n) + 2.0 ** -133).all()


@pytest.mark.parametrize("group", [0, 128])
def test_scales_that_round_to_zero(group):
    """A group whose scale is below fp32's smallest number has scale 0 and codes 0."""
    x = torch.zeros(1, 128)
    x[0, :4] = torch.tensor([2.0 ** -100, -(2.0 ** -101), 0.0, 2.0 ** -100])
    w = torch.full((128,), 2.0 ** -52)                             # n = 316 * 2^-152: two of fp32's smallest numbers
    x, w = x.bfloat16().cuda(), w.bfloat16().cuda()
    y8, sc = torch.full((1, 128), 3.0, device="cuda").to(torch.float8_e4m3fn), torch.full((1, 1), 7.0, device="cuda")
    abi.lora_rms_norm(x, w, 1e-5, y8=y8, scales=sc, group=group)
    assert (sc == 0).all() and (y8.float() == 0).all()
