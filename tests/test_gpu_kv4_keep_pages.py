"""lora_kv4_keep: a sequence whose rows one of the caches cannot move keeps its length."""
import numpy as np
import pytest
import torch

import draft_ref as R
from lora_serving_gb300 import abi, store
from test_gpu_kv4_keep import _built, _case  # noqa: F401

pytestmark = pytest.mark.gpu


def _keep(pages, table, q_lens, ctx, KV, D, page, n_keep, path, lens, n_pages=()):
    """n_pages: (cache, pages that it says it has)."""
    dev = torch.from_numpy(pages).cuda()
    layers = store.KV4Layers([store.KV4Cache(p.shape[0], page, KV, D, pages=p) for p in dev])
    for cache, n in n_pages:
        layers.c[cache].n_pages = n
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    abi.lora_kv4_keep(layers, store.KV4Batch.from_lens(q_lens, ctx, table), i32(n_keep), i32(path), lens=lens, dev_status=st)
    return dev.cpu().numpy(), abi.lora_read_device_status(st)


@pytest.mark.parametrize("layers,short", [(2, 0), (2, 1), (1, 0), (67, 2), (67, 66)])   # 67 caches are two launches
def test_a_cache_with_too_few_pages(layers, short):
    q_lens, ctx, KV, D, page = [6, 6, 6], [20, 40, 33], 1, 64, 16
    _, table, pages, _, _ = _case(7, q_lens, ctx, KV, D, page, layers, 6)
    need = [-(-c // page) for c in ctx]
    at = 1
    for s, n in enumerate(need):           # page 0 is nobody's: the short cache has no other
        table[s, :n] = np.arange(at, at + n)
        at += n
    path = np.array([[0, 2, 3], [1, 2, 5], [0, 1, 2]])          # the last one's rows are where they belong
    n_keep = np.array([3, 3, 3])
    lens = torch.full((3,), -3, dtype=torch.int32, device="cuda")
    got, st = _keep(pages, table, q_lens, ctx, KV, D, page, n_keep, path, lens, n_pages=[(short, 1)])
    assert st == abi.LORA_DEV_BAD_PAGE and lens.tolist() == [-3, -3, 30]
    for i in range(layers):
        assert np.array_equal(got[i], pages[i] if i == short else R.keep(pages[i], D, page, table, q_lens, ctx, n_keep, path))


def test_a_table_without_the_page():
    q_lens, ctx, KV, D, page = [6, 6], [20, 40], 2, 64, 16
    _, table, pages, _, _ = _case(8, q_lens, ctx, KV, D, page, 2, 6)
    path, n_keep = np.array([[0, 2, 3], [1, 2, 5]]), np.array([3, 3])
    for s, col in ((0, 1), (1, 2)):
        bad = table.copy()
        bad[s, col] = -1
        lens = torch.full((2,), -3, dtype=torch.int32, device="cuda")
        got, st = _keep(pages, bad, q_lens, ctx, KV, D, page, n_keep, path, lens)
        k = n_keep * (np.arange(2) != s)
        assert st == abi.LORA_DEV_BAD_PAGE and lens.tolist() == [-3 if i == s else c - n + 3 for i, (n, c) in enumerate(zip(q_lens, ctx))]
        assert all(np.array_equal(g, R.keep(p, D, page, table, q_lens, ctx, k, path)) for g, p in zip(got, pages))
