"""lora_kv4_attend and what its rows do not see: windows wider than any context."""
import math

import pytest
import torch

import kv4_ref as R
from lora_serving_gb300 import abi, build
from test_gpu_kv4 import BOUNDS, _attend, _close, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 5000])
@pytest.mark.parametrize("case", [([9, 1], [4, 300], 8, 2, 128, 64), ([3, 4], [0, 1], 6, 2, 64, 16), ([90, 65], [64, 500], 3, 1, 128, 64),
                                  ([300, 40], [7, 700], 8, 8, 64, 16)], ids=range(4))
def test_windows_wider_than_any_context(case, window, bounds):
    """With rows before the first position, from which a start this far back is not a number of 32 bits."""
    q_lens, ctx, H, KV, D, page = case
    q, K, V, table, cache, batch = _attend((*case, 0), 80 + H, bounds=bounds)
    scale = 1 / math.sqrt(D)
    got = _run(q, cache, batch, H, scale, window)
    assert torch.equal(got, _run(q, cache, batch, H, scale, 0))
    want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, q_lens, ctx, table, page, scale)
    _close(R.f64(got).reshape(-1, H, D), want, tol)
