"""lora_kv4_attend_tree against tests/draft_ref.py in 64 bits (the tolerance is derived in tests/kv4_ref.py)."""
import math

import numpy as np
import pytest
import torch

import draft_ref as R
import kv4_ref as K4
from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _table(rng, ctx, page, spare=2):
    need = [-(-c // page) for c in ctx]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(need), max([1, *need])), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


def _case(seed, q_lens, ctx, H, KV, D, page):
    rng = np.random.default_rng(seed)
    table, n_pages = _table(rng, ctx, page)
    pages = K4.random_pages(rng, n_pages, KV, page, D)
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), H * D)).astype(np.float32) * 2).bfloat16()
    return rng, table, pages, q


def _attend(q, pages, words, q_lens, ctx, table, H, KV, D, page, window=0, scale=None, out=None, stream=None, bounds=None):
    cache = store.KV4Cache(pages.shape[0], page, KV, D, pages=torch.from_numpy(pages).cuda())
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    if bounds:
        batch.c.max_q_len, batch.c.max_ctx_len = bounds
    ws = store.kv4_workspace(cache, H, batch)
    ws.fill_(255)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = q.cuda()
    out = torch.full_like(q, 7.0) if out is None else out
    abi.lora_kv4_attend_tree(out, q, cache, batch, torch.from_numpy(words).cuda(), ws, n_heads=H,
                             scale=1 / math.sqrt(D) if scale is None else scale, window=window, dev_status=st, stream=stream)
    return out, abi.lora_read_device_status(st)


CASES = [  # rows of each sequence, positions with them, heads, kv, D, page, window
    ([1], [1], 4, 4, 64, 16, 0),
    ([5], [5], 8, 2, 128, 16, 0),                                   # no context
    ([8], [1003], 32, 8, 128, 64, 0),
    ([7, 0, 1, 3], [7, 40, 33, 99], 6, 2, 128, 16, 0),
    ([4, 6, 2], [300, 17, 1000], 4, 4, 64, 32, 0),
    ([33], [70], 2, 1, 128, 16, 0),                                 # bits in two words, the tree across pages and tiles
    ([64, 10], [64, 500], 8, 8, 64, 64, 0),
    ([64, 20, 1], [700, 2100, 130], 32, 8, 128, 64, 0),             # many rows: tensor memory
    ([64, 31], [1500, 333], 16, 2, 128, 256, 0),                    # 512 rows of a kv head: two blocks of 256
    ([100, 129], [100, 1000], 8, 1, 64, 16, 0),                     # trees past 64 rows, and past a tile
    ([3, 40, 12], [4000, 900, 64], 24, 8, 128, 32, 0),
    ([5, 2], [400, 90], 8, 2, 128, 16, 40),                         # windows: inside a tile, across pages
    ([9, 30], [700, 45], 4, 4, 64, 16, 3),                          # narrower than the trees' depth
    ([64, 50], [1500, 100], 32, 8, 128, 64, 200),
    ([64, 64], [5000, 300], 16, 2, 64, 128, 1),
    ([16] * 12, [2000 + 37 * i for i in range(12)], 16, 2, 128, 64, 0),   # 128 rows of a kv head: both halves of the SM's tensor memory
    ([9, 16, 13, 32, 5, 16, 30], [1500, 257, 400, 3000, 129, 128, 140], 32, 4, 128, 64, 0),   # with items of 256 between them
    ([14] * 9, [700 + 61 * i for i in range(9)], 16, 2, 64, 16, 300),
    ([12], [9000], 8, 1, 128, 128, 0),                              # one item over many SMs
    ([6], [3], 4, 2, 128, 16, 0),                                   # rows before the first position
    ([60, 70], [30, 0], 8, 1, 128, 16, 20),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_tree(case, kind):
    q_lens, ctx, H, KV, D, page, window = case
    rng, table, pages, q = _case(sum(q_lens) + sum(ctx), q_lens, ctx, H, KV, D, page)
    if kind == "tree":
        bits = R.trees(rng, q_lens)
    else:   # any sets, rows without a bit among them
        bits = [[int.from_bytes(rng.bytes(-(-n // 8)), "little") & ((1 << n) - 1) if rng.random() < 0.8 else 0 for _ in range(n)] for n in q_lens]
    ld = -(-max(q_lens) // 32) + 1
    got, st = _attend(q, pages, R.words(bits, ld, rng), q_lens, ctx, table, H, KV, D, page, window)
    assert st == 0
    want, tol = R.attend_tree(K4.f64(q).reshape(-1, H, D), *K4.unpack(pages, page, D), bits, ctx, table, page, 1 / math.sqrt(D), window)
    err = np.abs(K4.f64(got).reshape(want.shape) - want)
    assert (err <= tol).all(), float((err - tol).max())
    size = np.linalg.norm(want, axis=-1)
    assert (np.linalg.norm(K4.f64(got).reshape(want.shape) - want, axis=-1) <= 2.0 ** -7 * size + 1e-12).all()


@pytest.mark.parametrize("case", [c for c in CASES if c[6] == 0 or c[6] >= max(c[0])], ids=str)
def test_chains_are_causal(case):
    """Rows that see all rows before them: lora_kv4_attend, bit for bit but for the cuts of long sums."""
    q_lens, ctx, H, KV, D, page, window = case
    rng, table, pages, q = _case(3, q_lens, ctx, H, KV, D, page)
    bits = R.trees(rng, q_lens, chain=True)
    got, _ = _attend(q, pages, R.words(bits, -(-max(q_lens) // 32)), q_lens, ctx, table, H, KV, D, page, window)
    cache = store.KV4Cache(pages.shape[0], page, KV, D, pages=torch.from_numpy(pages).cuda())
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    want = torch.full_like(got, 7.0)
    abi.lora_kv4_attend(want, q.cuda(), cache, batch, store.kv4_workspace(cache, H, batch), n_heads=H, scale=1 / math.sqrt(D), window=window)
    # each is within its own tolerance of the exact one: they differ by two bf16 half steps and the operands' rounding
    ref, tol = R.attend_tree(K4.f64(q).reshape(-1, H, D), *K4.unpack(pages, page, D), bits, ctx, table, page, 1 / math.sqrt(D), window)
    assert (np.abs(K4.f64(got) - K4.f64(want)).reshape(ref.shape) <= 2 * tol).all()


def _poison(pages, D, page, ids, off, value=np.nan):
    """Parameters of a position's K and V that make every value of it NaN or infinite."""
    for p, o in zip(ids, off):
        for h in range(pages.shape[1]):
            at = R.place_bytes(page, D, o)[D:]
            pages[p, h, at] = np.tile(np.array([value], "<f2").view(np.uint8), len(at) // 2)


@pytest.mark.parametrize("q_lens,ctx,H,KV,D,page", [([6, 5], [50, 37], 8, 2, 128, 16), ([64, 40], [300, 129], 32, 8, 128, 64),
                                                    ([9], [200], 4, 4, 64, 32), ([64], [90], 8, 1, 64, 16)], ids=str)
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_bytes_that_a_row_does_not_see(q_lens, ctx, H, KV, D, page, value):
    """A branch whose cached values are no numbers reaches the rows that see it and no other; so does nothing past the context."""
    rng, table, pages, q = _case(9, q_lens, ctx, H, KV, D, page)
    bits = R.trees(rng, q_lens)
    sick = [n // 2 for n in q_lens]
    used = np.zeros(pages.shape[:1] + (page,), bool)
    for s, c in enumerate(ctx):
        for j in range(c):
            used[table[s][j // page], j % page] = True
    clean = pages.copy()
    _poison(pages, D, page, *np.nonzero(~used), value)
    for s, (n, c) in enumerate(zip(q_lens, ctx)):
        j = c - n + sick[s]
        _poison(pages, D, page, [table[s][j // page]], [j % page], value)
    got, st = _attend(q, pages, R.words(bits, -(-max(q_lens) // 32)), q_lens, ctx, table, H, KV, D, page)
    want, tol = R.attend_tree(K4.f64(q).reshape(-1, H, D), *K4.unpack(clean, page, D), bits, ctx, table, page, 1 / math.sqrt(D))
    got = K4.f64(got).reshape(want.shape)
    sees = np.concatenate([[b >> sick[s] & 1 for b in mine] for s, mine in enumerate(bits)]).astype(bool)
    assert st == 0 and sees.any() and not sees.all()
    assert (np.abs(got[~sees] - want[~sees]) <= tol[~sees]).all()
    assert not np.isfinite(got[sees]).any()


def test_every_position_counts_once():
    """Under scale 0 each position that a row sees has the same weight, and leaves its own mark."""
    for q_lens, ctx, H, KV, D, page, window in (([20, 3], [150, 77], 8, 2, 128, 16, 0), ([64], [200], 16, 2, 64, 32, 0), ([2], [90], 4, 4, 64, 16, 30),
                                                ([40], [180], 8, 1, 128, 64, 50)):
        rng, table, pages, q = _case(4, q_lens, ctx, H, KV, D, page)
        bits = R.trees(rng, q_lens)
        G = D // 64
        vp = pages[:, :, page * (D + 4 * G):].view("<f2").reshape(*pages.shape[:2], page // 2, G, 2, 2)
        vp[..., 0, :] = 0
        vp[..., 1, :] = 0
        for s, c in enumerate(ctx):
            for j in range(c):      # V: 1 in the group of dims of the position's parity, elsewhere 0
                vp[table[s][j // page], :, j % page // 2, j % G, 1, j % 2] = 1.0 if G > 1 or j % 2 else 0.0
        got, _ = _attend(q, pages, R.words(bits, -(-max(q_lens) // 32)), q_lens, ctx, table, H, KV, D, page, window, scale=0.0)
        want, tol = R.attend_tree(K4.f64(q).reshape(-1, H, D), *K4.unpack(pages, page, D), bits, ctx, table, page, 0.0, window)
        # weights of 2^7 each, their sums and the marks exact: only the result is rounded
        assert (np.abs(K4.f64(got).reshape(want.shape) - want) <= 2.0 ** -8 * want + 1e-6).all()


def test_bad_pages_and_tables():
    q_lens, ctx, H, KV, D, page = [6, 40], [100, 80], 8, 2, 128, 16
    rng, table, pages, q = _case(2, q_lens, ctx, H, KV, D, page)
    bits = R.trees(rng, q_lens)
    words = R.words(bits, 2)
    bad = table.copy()
    bad[0, 2], bad[1, 4] = pages.shape[0], -3       # in the context; in the tree
    got, st = _attend(q, pages, words, q_lens, ctx, bad, H, KV, D, page)
    assert st == abi.LORA_DEV_BAD_PAGE
    Kf, Vf = K4.unpack(pages, page, D)
    gone = [set(range(32, 48)), set(range(64, 80))]
    # the same as rows that do not see the page: as bits over all positions of a context-free tree
    wide = [[int("".join("0" if (j in gone[s] or (j >= c - len(mine) and not mine[i] >> (j - c + len(mine)) & 1)) else "1" for j in reversed(range(c))), 2)
             for i in range(len(mine))] for s, (mine, c) in enumerate(zip(bits, ctx))]
    want, tol = np.zeros((sum(q_lens), H, D)), np.zeros((sum(q_lens), H, D))
    t = 0
    for s, (mine, c) in enumerate(zip(wide, ctx)):
        n = len(mine)
        qq = np.zeros((c, H, D))
        qq[c - n:] = K4.f64(q).reshape(-1, H, D)[t:t + n]
        o, e = R.attend_tree(qq, Kf, Vf, [[0] * (c - n) + mine], [c], table[s:s + 1], page, 1 / math.sqrt(D))
        want[t:t + n], tol[t:t + n] = o[c - n:], e[c - n:]
        t += n
    assert (np.abs(K4.f64(got).reshape(want.shape) - want) <= tol).all()
    # a sequence past the host's bounds is left alone
    got, st = _attend(q, pages, words, q_lens, ctx, table, H, KV, D, page, bounds=(40, 90))
    assert st == abi.LORA_DEV_BAD_SEGMENT and (got[:6] == 7).all() and not (got[6:] == 7).all(1).any()


def test_in_place_strides_stream_and_replay():
    q_lens, ctx, H, KV, D, page = [12, 64, 1], [300, 200, 40], 16, 4, 128, 32
    rng, table, pages, q = _case(6, q_lens, ctx, H, KV, D, page)
    bits = R.trees(rng, q_lens)
    want, _ = _attend(q, pages, R.words(bits, 2), q_lens, ctx, table, H, KV, D, page)
    wide = torch.full((sum(q_lens) + 3, H * D + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:-3, 8:8 + H * D] = q.cuda()
    view = wide[:-3, 8:8 + H * D]
    cache = store.KV4Cache(pages.shape[0], page, KV, D, pages=torch.from_numpy(pages).cuda())
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    ws = store.kv4_workspace(cache, H, batch)
    masks = torch.from_numpy(R.words(bits, 2)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi.lora_kv4_attend_tree(view, view, cache, batch, masks, ws, n_heads=H, scale=1 / math.sqrt(D), stream=side)
    side.synchronize()
    assert torch.equal(view, want) and (wide[-3:] == 5).all() and (wide[:, :8] == 5).all() and (wide[:, 8 + H * D:] == 5).all()
    # captured, then replayed with other trees
    out, qd = torch.zeros_like(want), q.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.lora_kv4_attend_tree(out, qd, cache, batch, masks, ws, n_heads=H, scale=1 / math.sqrt(D))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    other = R.words(R.trees(rng, q_lens), 2)
    masks.copy_(torch.from_numpy(other))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _attend(q, pages, other, q_lens, ctx, table, H, KV, D, page)[0]) and not torch.equal(out, want)
