"""The 4-bit cache's append, read and attention against plain references in
64 bits (tests/kv4_ref.py, where the tolerances are derived)."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as R
from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _table(rng, ctx_lens, page, spare=2):
    need = [-(-c // page) for c in ctx_lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(need), max([1, *need])), -1, np.int32)      # unused entries name no page
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append ----

APPENDS = [  # q_lens, ctx_lens, heads, kv, D, page, rot, pairs, positions
    ([1], [1], 4, 4, 64, 16, 64, [32], False),
    ([3, 0, 5, 1], [3, 40, 33, 17], 6, 2, 128, 16, 128, [64], False),
    ([17, 1, 64], [17, 100, 200], 8, 2, 128, 32, 128, [22, 21, 21], True),
    ([5, 9], [300, 9], 24, 8, 128, 256, 64, [20, 12], True),
    ([40], [41], 5, 1, 64, 64, 32, [7, 5, 4], True),
    ([2, 2, 2], [70, 2, 129], 3, 3, 64, 128, 0, [], False),
    ([33], [1000], 28, 4, 128, 64, 16, [8], True),
]


def _append(case, seed, x_scale=1.0, wide=0):
    q_lens, ctx, H, KV, D, page, rot, pairs, has_pos = case
    rng = np.random.default_rng(seed)
    T, W = sum(q_lens), (H + 2 * KV) * D
    x = torch.from_numpy((x_scale * rng.standard_normal((T, W + wide))).astype(np.float32)).bfloat16().cuda()
    table, n_pages = _table(rng, ctx, page)
    cache = store.KV4Cache(n_pages, page, KV, D)
    cache.pages.copy_(torch.from_numpy(rng.integers(0, 256, tuple(cache.pages.shape), dtype=np.uint8)))
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    rope = store.rope_table(max(ctx) + 5, rot // 2) if rot else None
    pos = rng.integers(0, max(ctx) + 5, (T, max(1, len(pairs)))).astype(np.int32) if has_pos else None
    return rng, x, table, cache, batch, rope, pos


@pytest.mark.parametrize("case", APPENDS, ids=range(len(APPENDS)))
def test_append_and_read(case):
    q_lens, ctx, H, KV, D, page, rot, pairs, has_pos = case
    rng, x, table, cache, batch, rope, pos = _append(case, 100 + D + H, wide=24)
    T = x.shape[0]
    before = cache.pages.cpu().numpy()
    q = torch.full((T, H * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    st = _status()
    abi.lora_kv4_append(q, x, cache, batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, rope=rope,
                        positions=None if pos is None else torch.from_numpy(pos).cuda(), axis_pairs=pairs or None,
                        dev_status=st)
    k, v = (torch.zeros(T, KV * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    abi.lora_kv4_read(k, v, cache, batch, dev_status=st)
    assert abi.lora_read_device_status(st) == 0
    after = cache.pages.cpu().numpy()

    where = R.places(q_lens, ctx)
    X = R.f64(x)[:, :(H + 2 * KV) * D].reshape(T, H + 2 * KV, D)
    at = np.array([[p] * max(1, len(pairs)) for _, p in where]) if pos is None else pos
    turned = X.copy()
    if rot:
        turned[:, :H + KV] = R.rotate(X[:, :H + KV], R.f64(rope), at, pairs)
    # q: one bf16 rounding of two fp32 products and a sum
    mag = np.abs(X[:, :H]).max()
    assert (np.abs(R.f64(q)[:, :H * D].reshape(T, H, D) - turned[:, :H]) <= 2.0 ** -8 * np.abs(turned[:, :H]) + 2.0 ** -21 * mag).all()
    assert (q[:, H * D:] == 7).all()
    # the bytes: exactly the stored form of the fp32 rotation
    t32 = X.astype(np.float32)
    if rot:
        tab = rope.cpu().numpy()
        i = np.arange(rot // 2)
        ax = np.repeat(np.arange(len(pairs)), pairs)
        c, s = (tab[at[:, ax], i, e][:, None] for e in (0, 1))
        lo, hi = t32[:, :H + KV, :rot // 2].copy(), t32[:, :H + KV, rot // 2:rot].copy()
        t32[:, :H + KV, :rot // 2], t32[:, :H + KV, rot // 2:rot] = lo * c - hi * s, hi * c + lo * s
    Kp, Vp = R.unpack(after, page, D)
    for name, got, new, pages in (("k", k, t32[:, H:H + KV], Kp), ("v", v, t32[:, H + KV:], Vp)):
        codes, step, low = R.quantise32(new)
        want = (codes.astype(np.float64) * step + low).reshape(T, KV, D)
        for t, (s, p) in enumerate(where):
            assert np.array_equal(pages[table[s][p // page], :, p % page], want[t]), (name, t)
        want32 = torch.from_numpy((codes * step + low).astype(np.float32).reshape(T, KV * D)).bfloat16()
        assert torch.equal(got.cpu(), want32), name
        # and the stored value is within half a step of the value, but for the fp16 roundings of the ends
        err = np.abs(want - (turned[:, H:H + KV] if name == "k" else X[:, H + KV:]))
        half = np.repeat(step[..., 0], 64, -1).reshape(T, KV, D) / 2
        assert (err <= half * (1 + 2.0 ** -8) + 2.0 ** -10 * np.abs(new).max()).all()
    # nothing else in the cache changed
    touched = np.zeros(after.shape, bool)
    G, ps = D // 64, page
    for s, p in where:
        o, b = p % page, touched[table[s][p // page]]
        b[:, o * D // 2:(o + 1) * D // 2] = True
        for wd in range(D // 4):
            base = ps * D // 2 + (o // 2) * D + 4 * wd + 2 * (o % 2)
            b[:, base:base + 2] = True
        b[:, ps * D + o * 4 * G:ps * D + (o + 1) * 4 * G] = True
        for g in range(G):
            base = ps * (D + 4 * G) + ((o // 2) * G + g) * 8 + 2 * (o % 2)
            b[:, base:base + 2] = True
            b[:, base + 4:base + 6] = True
    assert np.array_equal(after[~touched], before[~touched])


def test_append_rotates_in_place_and_skips_rows_without_a_place():
    H, KV, D, page = 4, 2, 128, 16
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, (H + 2 * KV) * D)).astype(np.float32)).bfloat16().cuda()
    keep = x.clone()
    cache = store.KV4Cache(3, page, KV, D)
    batch = store.KV4Batch.from_lens([4, 2], [2, 9], [[1], [0]])       # two of four rows stand before position 0
    rope = store.rope_table(16, 64)
    abi.lora_kv4_append(x[:, :H * D], x, cache, batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, rope=rope)
    want = R.rotate(R.f64(keep[:, :H * D]).reshape(6, H, D), R.f64(rope), np.array([[0], [0], [0], [1], [7], [8]]), [64])
    got = R.f64(x[:, :H * D]).reshape(6, H, D)
    assert torch.equal(x[:2], keep[:2]) and torch.equal(x[:, H * D:], keep[:, H * D:])
    assert (np.abs(got[2:] - want[2:]) <= 2.0 ** -8 * np.abs(want[2:]) + 2.0 ** -19).all()
    assert (cache.pages[2] == 0).all()


def test_append_extreme_values():
    """Constants, tiny ranges, saturation, infinities; a NaN stays in its group."""
    D, page, KV = 128, 16, 1
    x = torch.zeros(6, 3 * D, dtype=torch.bfloat16, device="cuda")
    x[0, D:] = 2.5
    x[1, D:2 * D] = torch.linspace(-1e-7, 1e-7, D)
    x[2, D:2 * D] = 1e38
    x[2, D] = -1e38
    x[3, D + 5] = float("inf")
    x[3, D + 6] = float("-inf")
    x[4, D + 70] = float("nan")
    x[5, 2 * D:] = torch.arange(D) * 1.0
    cache = store.KV4Cache(1, page, KV, D)
    batch = store.KV4Batch.from_lens([6], [6], [[0]])
    q = torch.empty(6, D, dtype=torch.bfloat16, device="cuda")
    abi.lora_kv4_append(q, x, cache, batch, n_heads=1, q_off=0, k_off=D, v_off=2 * D)
    K, V = (a[0, 0] for a in R.unpack(cache.pages.cpu().numpy(), page, D))
    assert (K[0] == 2.5).all() and (V[0] == 2.5).all()
    assert (np.abs(K[1]) <= 2e-7).all()
    sat = float(np.float16(60000.0))
    assert K[2, 0] == -sat and (np.abs(K[2, 1:64] - 60000) <= 15 * 2.0 ** -11 * 8000 + 32).all() and (K[2, 64:] == sat).all()
    assert np.isfinite(K[3]).all() and K[3, 5] > 59000 and K[3, 6] == -sat
    assert np.isnan(K[4, 64:]).all() and (K[4, :64] == 0).all()
    assert (np.abs(V[5] - np.arange(D)) <= 63 / 15 / 2 + 2.0 ** -11 * 64 + 63 * 2.0 ** -11).all()


def test_append_device_faults():
    H, KV, D, page = 2, 1, 64, 16
    x = torch.randn(4, (H + 2 * KV) * D, device="cuda").bfloat16()
    rope = store.rope_table(8, 32)
    q = torch.zeros(4, H * D, dtype=torch.bfloat16, device="cuda")
    args = dict(n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, rope=rope)

    def run(batch, cache, **more):
        st = _status()
        q.zero_()
        abi.lora_kv4_append(q, x, cache, batch, dev_status=st, **args, **more)
        return abi.lora_read_device_status(st)

    cache = store.KV4Cache(2, page, KV, D)
    assert run(store.KV4Batch.from_lens([4], [4], [[5]]), cache) == abi.LORA_DEV_BAD_PAGE
    assert (cache.pages == 0).all() and (q != 0).any(1).all()                 # q alone is written
    assert run(store.KV4Batch.from_lens([4], [4], [[-1]]), cache) == abi.LORA_DEV_BAD_PAGE
    pos = torch.tensor([[0], [7], [8], [-1]], dtype=torch.int32, device="cuda")
    assert run(store.KV4Batch.from_lens([4], [4], [[0]]), cache, positions=pos) == abi.LORA_DEV_BAD_POSITION
    assert (q != 0).any(1).tolist() == [True, True, False, False]
    low = store.KV4Batch.from_lens([2, 2], [3, 2], [[0], [1]])
    low.c.max_ctx_len = 2                                                      # the first sequence passes the bound
    assert run(low, cache) == abi.LORA_DEV_BAD_SEGMENT
    assert (q != 0).any(1).tolist() == [False, False, True, True]
    k, v = (torch.zeros(4, KV * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = _status()
    abi.lora_kv4_read(k, v, cache, store.KV4Batch.from_lens([4], [4], [[9]]), dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_PAGE and (k == 0).all() and (v == 0).all()


# ------------------------------------------------------------------ attend ----

ATTENDS = [  # q_lens, ctx_lens, heads, kv, D, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1], 32, 8, 128, 64, 0),
    ([1, 1, 1, 1, 1, 1], [15, 16, 17, 255, 256, 257], 8, 2, 128, 16, 0),
    ([1, 0, 1, 1], [0, 50, 1, 700], 24, 8, 128, 32, 0),
    ([1] * 9, [3, 1000, 31, 64, 65, 2, 129, 511, 90], 16, 4, 64, 128, 0),
    ([1], [4099], 8, 1, 128, 64, 0),
    ([1, 1, 1], [300, 1500, 77], 40, 8, 64, 256, 0),
    ([1, 1], [900, 513], 64, 4, 128, 16, 0),                       # 16 heads to a kv head
    ([1, 1], [700, 40], 64, 1, 64, 32, 0),                         # 64
    ([2, 5, 1, 3], [2, 77, 1000, 64], 8, 8, 128, 16, 0),
    ([4, 4], [500, 4], 16, 2, 128, 64, 0),                         # 32 query rows to a kv head
    ([7, 3], [257, 90], 12, 4, 64, 32, 0),
    ([1, 4, 1], [600, 333, 20], 8, 2, 128, 32, 64),                # windows inside a tile and across pages
    ([1, 3], [600, 333], 6, 2, 64, 16, 1),
    ([3, 9], [1, 5], 4, 4, 128, 16, 0),                            # rows before the first position
    ([33], [33], 8, 2, 128, 64, 0),                                # prompts
    ([128, 1, 70], [128, 400, 333], 8, 2, 128, 32, 0),
    ([129, 257], [129, 300], 6, 2, 128, 16, 0),
    ([200], [1111], 4, 1, 64, 128, 0),
    ([90, 65], [64, 500], 3, 1, 128, 64, 0),                       # 26 rows before the first position
    ([300, 40], [300, 700], 8, 8, 64, 16, 100),
    ([513], [513], 7, 1, 128, 256, 37),
]


# The host's bounds pick the kernel: exact ones send small batches to the
# kernel for few rows, a cluster to a unit; loose ones send up to 24 rows of a
# kv head to its form by ranges, more to the tensor-memory kernel.
BOUNDS = ["exact", "loose"]
LOOSE_CTX = 200000


def _attend(case, seed, q_scale=2.0, poison=True, bounds="exact"):
    q_lens, ctx, H, KV, D, page, window = case
    rng = np.random.default_rng(seed)
    table, n_pages = _table(rng, ctx, page)
    if bounds == "loose":
        wide = np.full((len(ctx), -(-LOOSE_CTX // page)), -1, np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    pages = R.random_pages(rng, n_pages, KV, page, D)
    K, V = R.unpack(pages, page, D)
    if poison:   # what no row may see: infinities and NaN in every masked place
        G = D // 64
        used = np.zeros((n_pages, page), bool)
        for s, c in enumerate(ctx):
            for p in range(c):
                used[table[s][p // page], p % page] = True
        for n in range(n_pages):
            for o in np.flatnonzero(~used[n]):
                kp = pages[n, :, page * D + o * 4 * G:page * D + (o + 1) * 4 * G]
                kp[:] = np.tile(np.array([np.nan, np.inf], "<f2").view(np.uint8), G)
                for g in range(G):
                    base = page * (D + 4 * G) + ((o // 2) * G + g) * 8 + 2 * (o % 2)
                    pages[n, :, base:base + 2] = np.array([np.inf], "<f2").view(np.uint8)
                    pages[n, :, base + 4:base + 6] = np.array([np.nan], "<f2").view(np.uint8)
    T = sum(q_lens)
    q = torch.from_numpy((q_scale * rng.standard_normal((T, H * D))).astype(np.float32)).bfloat16().cuda()
    cache = store.KV4Cache(n_pages, page, KV, D, pages=torch.from_numpy(pages).cuda())
    batch = store.KV4Batch.from_lens(q_lens, ctx, table)
    if bounds == "loose":
        batch.c.max_ctx_len = LOOSE_CTX
        batch.c.max_q_len += 3
    return q, K, V, table, cache, batch


def _run(q, cache, batch, H, scale, window=0, out=None):
    out = torch.full_like(q, 9.0) if out is None else out
    st = _status()
    ws = store.kv4_workspace(cache, H, batch)
    ws.fill_(0xFF)                                                 # a workspace holds anything
    abi.lora_kv4_attend(out, q, cache, batch, ws, n_heads=H, scale=scale, window=window, dev_status=st)
    assert abi.lora_read_device_status(st) == 0
    return out


def _close(got, want, tol):
    off = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (off <= tol).all(), (float((off / tol).max()), np.unravel_index(np.argmax(off / tol), off.shape))


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("case", ATTENDS, ids=range(len(ATTENDS)))
def test_attend(case, bounds):
    q_lens, ctx, H, KV, D, page, window = case
    q, K, V, table, cache, batch = _attend(case, 7 * H + D + len(ctx), bounds=bounds)
    scale = 1 / math.sqrt(D)
    got = R.f64(_run(q, cache, batch, H, scale, window)).reshape(-1, H, D)
    want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, q_lens, ctx, table, page, scale, window)
    _close(got, want, tol)
    for t, (_, p) in enumerate(R.places(q_lens, ctx)):
        if p < 0:
            assert (got[t] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 20])
def test_attend_many_short_sequences(D, window):
    """More blocks of query rows than SMs, several to each, most of them with
    nothing in the second tile of 128 rows, long runs of these between two
    that have both; short ones for the kernel for few rows among them."""
    q_lens = ([30] * 37 + [70] + [2] * 5 + [64, 33] + [31] * 40 + [90]) * 2
    ctx = [n + 7 * (i % 5) for i, n in enumerate(q_lens)]
    case = (q_lens, ctx, 32, 8, D, 32, window)
    q, K, V, table, cache, batch = _attend(case, 5 + D, bounds="exact")
    got = R.f64(_run(q, cache, batch, 32, 0.1, window)).reshape(-1, 32, D)
    want, tol = R.attend(R.f64(q).reshape(-1, 32, D), K, V, q_lens, ctx, table, 32, 0.1, window)
    _close(got, want, tol)


@pytest.mark.parametrize("q_len", [1, 4, 40])
@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("bounds", BOUNDS)
def test_attend_scales(q_len, scale, bounds):
    """No score at all, a negative scale, and scores in the hundreds (one position takes all the weight)."""
    case = ([q_len, q_len], [300, 131], 8, 2, 128, 32, 0)
    q, K, V, table, cache, batch = _attend(case, 5, bounds=bounds)
    got = R.f64(_run(q, cache, batch, 8, scale)).reshape(-1, 8, 128)
    want, tol = R.attend(R.f64(q).reshape(-1, 8, 128), K, V, case[0], case[1], table, 32, scale)
    _close(got, want, tol)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("q_len", [1, 50])
def test_attend_query_range(q_len, bounds):
    """Rows of zeros, and rows whose values lie outside fp16's range."""
    case = ([q_len, q_len], [200, 96], 4, 2, 64, 16, 0)
    q, K, V, table, cache, batch = _attend(case, 6, q_scale=1.0, bounds=bounds)
    q[0, :64] = 0
    q[0, 64:128] *= 1e-7
    q[0, 128:192] *= 1e6
    for scale, h in ((0.1, 0), (1e6, 1), (1e-7, 2)):
        got = R.f64(_run(q, cache, batch, 4, scale)).reshape(-1, 4, 64)[:1, h]
        want, tol = R.attend(R.f64(q).reshape(-1, 4, 64), K, V, case[0], case[1], table, 16, scale)
        _close(got, want[:1, h], tol[:1, h])


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 1, 2], [60, 1, 45]])
def test_attend_strides_alias_and_far_pages(q_lens, bounds):
    """q and out as slices of wider rows, out over q, and pages a gigabyte apart (offsets past 32 bits)."""
    ctx, H, KV, D, page = [130, 64, 99], 8, 2, 128, 32
    case = (q_lens, ctx, H, KV, D, page, 0)
    q, K, V, table, cache, batch = _attend(case, 8, bounds=bounds)
    n, kv, block = cache.pages.shape
    gap = 700 * 1024 * 1024
    big = torch.empty((n - 1) * gap + kv * block, dtype=torch.uint8, device="cuda")
    far = torch.as_strided(big, (n, kv, block), (gap, block, 1))
    far.copy_(cache.pages)
    assert (n - 1) * gap > 1 << 32
    cache2 = store.KV4Cache(n, page, KV, D, pages=far)
    wide = torch.full((q.shape[0], H * D + 72), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 24:24 + H * D] = q
    view = wide[:, 24:24 + H * D]
    scale = 1 / math.sqrt(D)
    plain = _run(q, cache, batch, H, scale)
    _run(view, cache2, batch, H, scale, out=view)
    assert torch.equal(view, plain)
    assert (wide[:, :24] == 3).all() and (wide[:, 24 + H * D:] == 3).all()
    want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, q_lens, ctx, table, page, scale)
    _close(R.f64(plain).reshape(-1, H, D), want, tol)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("q_len", [1, 60])
def test_attend_repeats_bit_for_bit_and_on_another_stream(q_len, bounds):
    case = ([q_len] * 5, [3000, 60, 1, 800, 1999], 16, 4, 128, 64, 0)
    q, K, V, table, cache, batch = _attend(case, 9, bounds=bounds)
    first = _run(q, cache, batch, 16, 0.1)
    ws = store.kv4_workspace(cache, 16, batch)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(q) for _ in range(20)]
    for o in outs:
        abi.lora_kv4_attend(o, q, cache, batch, ws, n_heads=16, scale=0.1, stream=st)
    st.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_attend_graph_replay_with_refilled_tables():
    """A captured step keeps serving as its requests grow."""
    H, KV, D, page = 8, 2, 128, 16
    case = ([1, 1], [40, 100], H, KV, D, page, 0)
    q, K, V, table, cache, batch = _attend(([1, 1], [400, 300], H, KV, D, page, 0), 10, poison=False)
    full = batch.block_table.cpu().numpy()
    ws, out = store.kv4_workspace(cache, H, batch), torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        abi.lora_kv4_attend(out, q, cache, batch, ws, n_heads=H, scale=0.1)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.lora_kv4_attend(out, q, cache, batch, ws, n_heads=H, scale=0.1)
    for ctx in ([1, 2], [400, 300], [16, 0], [399, 17]):
        batch.ctx_lens.copy_(torch.tensor(ctx, dtype=torch.int32))
        g.replay()
        want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, case[0], ctx, full, page, 0.1)
        _close(R.f64(out).reshape(-1, H, D), want, tol)


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("q_len", [1, 4, 70])
def test_attend_device_faults(q_len, bounds):
    H, KV, D, page = 4, 2, 64, 16
    case = ([q_len, q_len, q_len], [200, 96, 130], H, KV, D, page, 0)
    q, K, V, table, cache, batch = _attend(case, 11, bounds=bounds)
    ws, st = store.kv4_workspace(cache, H, batch), _status()
    clean = _run(q, cache, batch, H, 0.1)
    rows = [slice(i * q_len, (i + 1) * q_len) for i in range(3)]
    # a page that the cache does not have: its positions are masked, the other sequences unchanged
    batch.block_table[1, 1] = 10 ** 6
    out = torch.full_like(q, 5.0)
    abi.lora_kv4_attend(out, q, cache, batch, ws, n_heads=H, scale=0.1, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_PAGE
    assert torch.equal(out[rows[0]], clean[rows[0]]) and torch.equal(out[rows[2]], clean[rows[2]])
    assert out[rows[1]].isfinite().all()
    K2, V2 = K.copy(), V.copy()
    t = R.f64(q).reshape(-1, H, D)[rows[1]]
    keep = np.r_[0:16, 32:96]
    pg = batch.block_table[1].cpu().numpy()
    k = np.concatenate([K2[p] for p in (pg[0], *pg[2:6])], 1)
    v = np.concatenate([V2[p] for p in (pg[0], *pg[2:6])], 1)
    i = q_len - 1                                                  # the last row sees all that is left
    for h in range(KV):
        sc = 0.1 * t[i, 2 * h:2 * h + 2] @ k[h].T
        w = np.exp(sc - sc.max(1, keepdims=True))
        o = (w / w.sum(1, keepdims=True)) @ v[h]
        assert len(keep) == k.shape[1]
        assert np.abs(R.f64(out).reshape(-1, H, D)[rows[1]][i, 2 * h:2 * h + 2] - o).max() < 0.05
    # a sequence above the host's bounds: its rows are not written
    st.zero_()
    batch.block_table[1, 1] = int(table[1, 1])
    batch.ctx_lens[2] = 10 ** 7
    out.fill_(5.0)
    abi.lora_kv4_attend(out, q, cache, batch, ws, n_heads=H, scale=0.1, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    assert (out[rows[2]] == 5).all()
    # the others' work is cut into other ranges without it: right within the tolerance, not bit for bit
    want, tol = R.attend(R.f64(q).reshape(-1, H, D), K, V, case[0], case[1], table, page, 0.1)
    _close(R.f64(out).reshape(-1, H, D)[:2 * q_len], want[:2 * q_len], tol[:2 * q_len])


@pytest.mark.parametrize("bounds", BOUNDS)
@pytest.mark.parametrize("part", ["k", "v"])
@pytest.mark.parametrize("q_len", [1, 3, 40, 150])
def test_attend_nan_reaches_the_rows_that_see_it(q_len, part, bounds):
    """A NaN in one position's K or V of one kv head (of V, in one group of dims): rows that see the position get
    NaN (in those dims), the others are as without it."""
    D, page, n_kv = 128, 16, 2
    case = ([q_len, 2], [q_len + 70, 90], 4, n_kv, D, page, 0)
    q, K, V, table, cache, batch = _attend(case, 12, bounds=bounds)
    clean = _run(q, cache, batch, 4, 0.1).view(-1, 4, D)
    at = 70 + q_len // 2                                          # seen by the rows from q_len // 2 on
    o = at % page
    off = page * D + o * 8 + 4 if part == "k" else page * (D + 8) + (o // 2) * 16 + 8 + 2 * (o % 2)      # group 1 of K, of V
    for low in (0, 2 if part == "k" else 4):
        cache.pages[int(table[0, at // page]), 1, off + low:off + low + 2] = torch.tensor([0, 0x7E], dtype=torch.uint8)
    out = _run(q, cache, batch, 4, 0.1).view(-1, 4, D)
    sees = torch.zeros(q_len + 2, 4, D, dtype=torch.bool, device="cuda")
    sees[q_len // 2:q_len, 2:, (64 if part == "v" else 0):] = True
    assert torch.equal(out.isnan(), sees)
    assert torch.equal(out[~sees], clean[~sees])


def test_python_calls_check_their_tensors():
    """What would make a kernel read or write past a tensor, or another type,
    is refused before anything is enqueued; raw status pointers pass."""
    H, KV, D, page = 4, 2, 128, 32
    cache = store.KV4Cache(4, page, KV, D)
    batch = store.KV4Batch.from_lens([3, 1], [3, 40], [[0, 1], [2, 3]])
    T, W = 4, (H + 2 * KV) * D
    x, q = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H * D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(T, KV * D, dtype=torch.bfloat16, device="cuda")
    rope = store.rope_table(64, D // 2)
    pos = torch.zeros(T, 3, dtype=torch.int32, device="cuda")
    ws = store.kv4_workspace(cache, H, batch)
    st = _status()
    n0 = abi.lora_kernel_launch_count()

    def append(**c):
        v = dict(q=q, x=x, rope=rope, positions=pos, axis_pairs=(20, 20, 24), dev_status=st) | c
        abi.lora_kv4_append(v.pop("q"), v.pop("x"), cache, batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, **v)

    bad = [lambda: append(q=q[:3]), lambda: append(q=q[:, :-8]), lambda: append(q=q.float()), lambda: append(q=q.t()), lambda: append(q=q[0]),
           lambda: append(x=x.half()), lambda: append(x=x[:2]), lambda: append(rope=rope.double()), lambda: append(rope=rope[:, ::2]),
           lambda: append(rope=rope[..., 0]), lambda: append(positions=pos.long()), lambda: append(positions=pos[:, :2]),
           lambda: append(axis_pairs=(16, 16, 16, 16)), lambda: append(axis_pairs=()), lambda: append(dev_status=st.float()),
           lambda: abi.lora_kv4_read(k, k[:3], cache, batch), lambda: abi.lora_kv4_read(k[:, ::2], k, cache, batch),
           lambda: abi.lora_kv4_attend(q, q[:, :-D], cache, batch, ws, n_heads=H, scale=0.1),
           lambda: abi.lora_kv4_attend(q, q, cache, batch, ws.cpu(), n_heads=H, scale=0.1),
           lambda: abi.lora_rms_norm(x, torch.ones(W, device="cuda"), 1e-5, y=x),
           lambda: abi.lora_rms_norm(x, x[0].clone(), 1e-5, y=x[:3]),
           lambda: abi.lora_rms_norm(x, x[0].clone(), 1e-5, y8=x.to(torch.float8_e4m3fn), scales=torch.ones(T, W // 128 - 1, device="cuda"), group=128)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    assert abi.lora_kernel_launch_count() == n0
    append(dev_status=st.data_ptr())
    append(rope=None, dev_status=None)
    append(axis_pairs=[20, 20, 24], positions=pos[:, :])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    abi.lora_kv4_attend(q, q, cache, batch, ws, n_heads=H, scale=0.1, dev_status=st, stream=s)
    abi.lora_kv4_attend(q, q, cache, batch, ws, n_heads=H, scale=0.1, dev_status=st, stream=s.cuda_stream)
    s.synchronize()
    assert abi.lora_read_device_status(st) == 0
