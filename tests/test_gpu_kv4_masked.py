"""lora_kv4_attend and what its rows do not see: positions behind a window and
ahead of a row, whatever their bytes, pages that were given back, windows
wider than any context."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as R
from lora_serving_gb300 import abi, build, store
from test_gpu_kv4 import BOUNDS, _attend, _close, _run, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _poison_v(pages, page, D, n, o, step, low):
    """The parameters of V at offset o of page n, every head and group."""
    for g in range(D // 64):
        at = page * (D + 4 * (D // 64)) + ((o // 2) * (D // 64) + g) * 8 + 2 * (o % 2)
        pages[n, :, at:at + 2] = np.array([step], "<f2").view(np.uint8)
        pages[n, :, at + 4:at + 6] = np.array([low], "<f2").view(np.uint8)


def _poison_k(pages, page, D, n, o, step, low):
    at = page * D + o * 4 * (D // 64)
    pages[n, :, at:at + 4 * (D // 64)] = np.tile(np.array([step, low], "<f2").view(np.uint8), D // 64)


# (step, low): not finite, and finite ones whose values leave fp16
BYTES = [(np.nan, np.inf), (60000.0, 0.0), (-65504.0, 65504.0), (4400.0, 30000.0), (0.0, -np.inf)]
WINDOWED = [  # q_lens, ctx_lens, heads, kv, D, page, window
    ([1], [5000], 8, 2, 128, 64, 1000),
    ([1, 1, 2], [300, 90, 700], 8, 2, 128, 16, 40),
    ([3, 1], [601, 333], 12, 4, 64, 32, 77),
    ([40, 33], [400, 999], 8, 2, 128, 16, 100),
    ([70, 130], [500, 1300], 8, 8, 64, 256, 333),
    ([150], [1150], 16, 2, 128, 128, 517),
]


def _first_seen(n, c, window):
    return max(0, c - n - window + 1)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("case", WINDOWED, ids=range(len(WINDOWED)))
def test_bytes_behind_the_window(case, bounds):
    q_lens, ctx, H, KV, D, page, window = case
    q, K, V, table, cache, batch = _attend(case, 40 + H + D, bounds=bounds)
    scale = 1 / math.sqrt(D)
    clean = _run(q, cache, batch, H, scale, window)
    want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, q_lens, ctx, table, page, scale, window)
    _close(R.f64(clean).reshape(-1, H, D), want, tol)
    keep = cache.pages.cpu().numpy()
    for step, low in BYTES:
        pages = keep.copy()
        for s, (n, c) in enumerate(zip(q_lens, ctx)):
            for p in range(_first_seen(n, c, window)):
                _poison_k(pages, page, D, table[s][p // page], p % page, step, low)
                _poison_v(pages, page, D, table[s][p // page], p % page, step, low)
        cache.pages.copy_(torch.from_numpy(pages))
        assert torch.equal(_run(q, cache, batch, H, scale, window), clean), (step, low)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("q_len", [2, 5, 40, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_bytes_ahead_of_a_row(q_len, D, bounds):
    """V of the last positions, which only the last rows see: the others are as they were."""
    H, KV, page = 4, 2, 16
    case = ([q_len, q_len], [q_len + 170, q_len], H, KV, D, page, 0)
    q, K, V, table, cache, batch = _attend(case, 60 + q_len, bounds=bounds)
    clean = _run(q, cache, batch, H, 0.1).view(2, q_len, -1)
    keep = cache.pages.cpu().numpy()
    last = max(1, q_len // 3)
    for step, low in BYTES:
        pages = keep.copy()
        for s, c in enumerate(case[1]):
            for p in range(c - last, c):
                _poison_v(pages, page, D, table[s][p // page], p % page, step, low)
        cache.pages.copy_(torch.from_numpy(pages))
        got = _run(q, cache, batch, H, 0.1).view(2, q_len, -1)
        assert torch.equal(got[:, :q_len - last], clean[:, :q_len - last]), (step, low)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [2, 1, 4], [60, 1, 33]])
def test_pages_given_back_behind_the_window(q_lens, page, bounds):
    """A table may name any page, or none, where no row sees a position."""
    H, KV, D = 8, 2, 128
    for ctx, window in (([1000, 600, 300], 100), ([733, 1290, 65], 17), ([2000, 90, 1111], 512), ([999, 1001, 1003], 1)):
        case = (q_lens, ctx, H, KV, D, page, window)
        q, K, V, table, cache, batch = _attend(case, page + window, bounds=bounds)
        clean = _run(q, cache, batch, H, 0.1, window)
        for none in (-1, 10 ** 6):
            for s, (n, c) in enumerate(zip(q_lens, ctx)):
                batch.block_table[s, :_first_seen(n, c, window) // page] = none
            assert torch.equal(_run(q, cache, batch, H, 0.1, window), clean)        # (and no status)


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


def test_tables_that_decrease():
    """The kernel for many rows leaves its sequences out of a batch whose q_starts decrease: together they could have more
    rows than the batch, and more tiles than its bounds allow."""
    H, KV, D, page = 8, 2, 128, 32
    q, K, V, table, cache, batch = _attend(([60, 50, 90], [100, 300, 200], H, KV, D, page, 0), 90, bounds="loose")
    batch.q_starts.copy_(torch.tensor([0, 60, 20, 110], dtype=torch.int32))
    out, st = torch.full_like(q, 5.0), _status()
    abi.lora_kv4_attend(out, q, cache, batch, store.kv4_workspace(cache, H, batch), n_heads=H, scale=0.1, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    assert (out == 5).all()
