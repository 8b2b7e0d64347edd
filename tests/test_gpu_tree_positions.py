"""lora_kv4_attend_tree counts every position that a row sees once, and no other: caches in which each position leaves its
own mark (tree_positions.py); what this catches is in test_tree_positions_host.py."""
import numpy as np
import pytest
import torch

import draft_ref as R
import kv4_positions as P
import kv4_ref as K4
import tree_positions as T
from lora_serving_gb300 import abi, build, store
from test_gpu_kv4 import BOUNDS, LOOSE_CTX, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("case", T.CASES, ids=range(len(T.CASES)))
def test_every_position_once(case, kind, bounds):
    q_lens, ctx, H, KV, D, page, window = case
    rng = np.random.default_rng(len(ctx) + D)
    table, n_pages = _table(rng, ctx, page)
    pages = P.pages_of(case, rng, table, n_pages)
    if bounds == "loose":
        wide = np.full((len(ctx), -(-LOOSE_CTX // page)), -1, np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    cache = store.KV4Cache(n_pages, page, KV, D, pages=torch.from_numpy(pages).cuda())
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    if bounds == "loose":
        batch.c.max_ctx_len = LOOSE_CTX
    bits = T.bits_of(case, kind)
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), H * D)).astype(np.float32)).bfloat16().cuda()
    words = torch.from_numpy(R.words(bits, -(-max(q_lens) // 32), rng)).cuda()
    out, st = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_kv4_attend_tree(out, q, cache, batch, words, store.kv4_workspace(cache, H, batch), n_heads=H, scale=0.0, window=window, dev_status=st)
    assert abi.lora_read_device_status(st) == 0
    assert P.off_by(K4.f64(out).reshape(-1, H, D), T.want(case, T.seen(case, bits))) <= 1
