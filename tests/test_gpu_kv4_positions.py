"""lora_kv4_attend counts every position that a row sees once, and no other:
caches in which each position leaves its own mark (kv4_positions.py), and the
relative error of whole rows.  What these catch, and how far a position or a
tile left out would move them, is in test_kv4_positions_host.py."""
import math

import numpy as np
import pytest
import torch

import kv4_positions as P
import kv4_ref as R
from lora_serving_gb300 import abi, build, store
from test_gpu_kv4 import ATTENDS, BOUNDS, LOOSE_CTX, _attend, _run, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("case", P.CASES, ids=range(len(P.CASES)))
def test_every_position_once(case, bounds):
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
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), H * D)).astype(np.float32)).bfloat16().cuda()
    got = R.f64(_run(q, cache, batch, H, 0.0, window)).reshape(-1, H, D)
    assert P.off_by(got, P.want(case)) <= 1


# The result in bf16 costs at most 2^-8 of a row, weights and values in fp16 2^-11 each, and the scores, of a standard
# deviation of three, 2^-10: q and the keys in fp16 cost each of their 64 or 128 products up to 2^-11, with either sign.
REL = 2.0 ** -7
LONG = [([1, 1, 1], [30000, 9000, 777], 32, 8, 128, 64, 0), ([40, 20], [5000, 900], 16, 4, 128, 32, 0), ([3, 2], [6000, 12000], 8, 8, 64, 16, 4096)]


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("case", ATTENDS + LONG, ids=range(len(ATTENDS + LONG)))
def test_relative_error_of_rows(case, bounds):
    q_lens, ctx, H, KV, D, page, window = case
    q, K, V, table, cache, batch = _attend(case, 3 * H + D + len(ctx), bounds=bounds)
    scale = 1 / math.sqrt(D)
    got = R.f64(_run(q, cache, batch, H, scale, window)).reshape(-1, H, D)
    want, _ = R.attend(R.f64(q).reshape(-1, H, D), K, V, q_lens, ctx, table, page, scale, window)
    off, size = np.linalg.norm(got - want, axis=2), np.linalg.norm(want, axis=2)
    assert (off <= REL * size).all(), float((off / size)[size > 0].max())
