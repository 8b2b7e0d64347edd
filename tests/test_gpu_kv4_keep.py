"""lora_kv4_keep against tests/draft_ref.py: bytes, all equal."""
import numpy as np
import pytest
import torch

import draft_ref as R
from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _case(seed, q_lens, ctx, KV, D, page, layers, columns):
    rng = np.random.default_rng(seed)
    need = [-(-c // page) for c in ctx]
    table = np.full((len(ctx), max([1, *need])), -1, np.int32)
    ids, at = rng.permutation(sum(need) + 2), 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    pages = rng.integers(0, 256, (layers, len(ids), KV, page * (D + 8 * (D // 64))), dtype=np.uint8)
    n_keep = np.array([rng.integers(0, min(n, columns) + 1) for n in q_lens])
    path = rng.integers(-9, 99, (len(ctx), columns))        # what lies behind a path's end does not matter
    for s, k in enumerate(n_keep):
        path[s, :k] = np.sort(rng.permutation(q_lens[s])[:k])
    return rng, table, pages, n_keep, path


def _keep(pages, table, q_lens, ctx, KV, D, page, n_keep, path, lens=None, n_pages=None, stream=None):
    dev = torch.from_numpy(pages).cuda()
    layers = store.KV4Layers([store.KV4Cache(p.shape[0], page, KV, D, pages=p) for p in dev])
    if n_pages is not None:
        layers.c[0].n_pages = n_pages
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    batch, k, p = store.KV4Batch.from_lens(q_lens, ctx, table), i32(n_keep), i32(path)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    abi.lora_kv4_keep(layers, batch, k, p, lens=lens, dev_status=st, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return dev.cpu().numpy(), abi.lora_read_device_status(st)


CASES = [  # rows, positions with them, kv, D, page, layers, columns of path
    ([1], [1], 1, 64, 16, 1, 1),
    ([7], [9], 2, 128, 16, 1, 7),
    ([16], [1000], 8, 128, 64, 28, 4),
    ([5, 0, 40, 1], [5, 33, 70, 100], 3, 64, 32, 3, 40),          # more than a warp's lanes, across pages
    ([64, 64, 64], [64, 200, 333], 8, 128, 16, 2, 64),
    ([130], [300], 9, 128, 256, 1, 100),
    ([12, 9], [500, 40], 1, 128, 128, 67, 12),                    # two launches
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("seed", [0, 1])
def test_keep(case, seed):
    q_lens, ctx, KV, D, page, layers, columns = case
    rng, table, pages, n_keep, path = _case(seed, q_lens, ctx, KV, D, page, layers, columns)
    lens = torch.full((len(ctx),), -3, dtype=torch.int32, device="cuda")
    got, st = _keep(pages, table, q_lens, ctx, KV, D, page, n_keep, path, lens, stream=torch.cuda.Stream() if seed else None)
    assert st == 0
    for p, want in zip(got, pages):
        assert np.array_equal(p, R.keep(want, D, page, table, q_lens, ctx, n_keep, path))
    assert lens.tolist() == [c - n + k for n, c, k in zip(q_lens, ctx, n_keep)]


def test_moves_that_follow_each_other():
    """Every place but the first is both read and written."""
    n, page, KV, D = 64, 16, 2, 128
    _, table, pages, _, _ = _case(3, [n], [n + 5], KV, D, page, 1, n)
    for path in ([0, *range(2, n)], list(range(1, n)), list(range(n)), [n - 1], [0, n - 1]):
        p = np.zeros((1, n), np.int64)
        p[0, :len(path)] = path
        got, st = _keep(pages, table, [n], [n + 5], KV, D, page, [len(path)], p)
        assert st == 0 and np.array_equal(got[0], R.keep(pages[0], D, page, table, [n], [n + 5], [len(path)], p))


def test_faults():
    q_lens, ctx, KV, D, page = [6, 6, 6, 6, 6, 9], [20, 40, 33, 6, 50, 4], 2, 64, 16
    _, table, pages, _, _ = _case(4, q_lens, ctx, KV, D, page, 2, 6)
    path = np.tile([0, 2, 3, 5, 0, 0], (6, 1))
    n_keep = np.array([3, 3, 3, 3, 3, 3])

    def run(change=None, **more):
        p, k = path.copy(), n_keep.copy()
        if change:
            change(p, k)
        lens = torch.full((6,), -3, dtype=torch.int32, device="cuda")
        got, st = _keep(pages, table if "table" not in more else more["table"], q_lens, ctx, KV, D, page, k, p, lens, more.get("n_pages"))
        return got, st, lens.tolist()

    want = [R.keep(p, D, page, table, q_lens, ctx, n_keep, path) for p in pages]
    whole = [17, 37, 30, 3, 47, -3]                    # the last one has no place: neither moved nor counted
    got, st, lens = run()
    assert st == 0 and np.array_equal(got, want) and lens == whole

    def as_if_none(s):
        k = n_keep.copy()
        k[s] = 0
        return [R.keep(p, D, page, table, q_lens, ctx, k, path) for p in pages]

    top = 2 ** 31 - 1
    for at, v, bit in ((("k", 1), 7, abi.LORA_DEV_BAD_SEGMENT), (("k", 1), -1, abi.LORA_DEV_BAD_SEGMENT), (("k", 1), top, abi.LORA_DEV_BAD_SEGMENT),
                       (("p", 1, 0), -1, abi.LORA_DEV_BAD_POSITION), (("p", 1, 1), 0, abi.LORA_DEV_BAD_POSITION), (("p", 1, 2), 6, abi.LORA_DEV_BAD_POSITION),
                       (("p", 1, 2), top, abi.LORA_DEV_BAD_POSITION), (("p", 1, 1), -top, abi.LORA_DEV_BAD_POSITION), (("p", 1, 2), 2, abi.LORA_DEV_BAD_POSITION)):
        def change(p, k):
            if at[0] == "k":
                k[at[1]] = v
            else:
                p[at[1:]] = v
        got, st, lens = run(change)
        assert st == bit and np.array_equal(got, as_if_none(1)) and lens == [*whole[:1], -3, *whole[2:]], (at, v)
    bad = table.copy()
    bad[2, 1] = -1                                     # its positions 27..32: the moves' pages
    got, st, _ = run(table=bad)
    assert st == abi.LORA_DEV_BAD_PAGE and np.array_equal(got, as_if_none(2))
    got, st, _ = run(n_pages=1)                        # the first cache has one page only; the other moves
    assert st == abi.LORA_DEV_BAD_PAGE and np.array_equal(got[1], want[1])
