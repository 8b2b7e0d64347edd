"""lora_kv4_plan against tests/draft_ref.py: whole numbers, all equal."""
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


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _state(rng, n, page, max_ctx, spare, ended=0.1, idle=0.1, q_max=4, extra=1):
    lens = rng.integers(0, max(1, max_ctx - q_max + 1), n)
    q = np.where(rng.random(n) < ended, -1, np.where(rng.random(n) < idle, 0, rng.integers(1, q_max + 1, n)))
    held = np.minimum(-(-lens // page) + rng.integers(0, extra + 1, n), -(-max_ctx // page))
    ids = rng.permutation(int(held.sum()) + spare)
    table = np.full((n, -(-max_ctx // page)), -1, np.int64)
    at = 0
    for s in range(n):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    free = np.concatenate([ids[at:], np.full(at, -7)])
    return dict(q=q, lens=lens, held=held, table=table, free=free, n_free=spare)


def _run(st, *, page, max_rows, max_q, max_ctx, depths=None, in_place=False, stream=None):
    more = {} if in_place else dict(n_free_out=torch.full((1,), -5, dtype=torch.int32, device="cuda"),
                                    held_out=torch.full((max(1, len(st["held"])),), -5, dtype=torch.int32, device="cuda")[:len(st["held"])])
    p = store.KV4Plan(_i32(st["free"]), _i32([st["n_free"]]), _i32(st["held"]), _i32(st["table"]), page_size=page, max_rows=max_rows,
                      max_q_len=max_q, max_ctx_len=max_ctx, **more)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_i32(st["q"]), _i32(st["lens"]))
    for t in (p.q_starts, p.ctx_lens, p.row_seq, p.slots):   # what was there does not matter
        t.fill_(77)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    abi.lora_kv4_plan(p, *args, depths=None if depths is None else _i32(depths), dev_status=word, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return p, args, word


def _check(p, word, want, faults):
    got = dict(q_starts=p.q_starts, ctx_lens=p.ctx_lens, block_table=p.block_table, held=p.held_out, free_pages=p.free_pages,
               row_seq=p.row_seq, positions=p.positions[:, 0], slots=p.slots)
    for k, t in got.items():
        assert np.array_equal(t.cpu().numpy().astype(np.int64), want[k]), k
    assert int(p.n_free_out) == want["n_free"]
    assert abi.lora_read_device_status(word) == faults


CASES = [  # sequences, page, longest context, spare pages, most rows of a sequence, rows more than there are
    (1, 16, 40, 5, 1, 0), (1, 64, 64, 0, 3, 7), (5, 16, 33, 2, 4, 0), (64, 64, 4096, 64, 1, 0), (31, 256, 1000, 4, 64, 100),
    (300, 32, 500, 40, 5, 3), (1025, 128, 3000, 900, 4, 0), (4096, 16, 200, 700, 16, 11), (256, 64, 2000, 2000, 700, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_plan(case, in_place):
    n, page, max_ctx, spare, q_max, more = case
    rng = np.random.default_rng(n + page)
    st = _state(rng, n, page, max_ctx, spare, q_max=min(q_max, max_ctx))
    rows = int(np.maximum(st["q"], 0).sum()) + more
    depths = rng.integers(-1, 9, rows) if n % 2 else None
    kw = dict(page=page, max_rows=rows, max_q=q_max, max_ctx=max_ctx, depths=depths)
    want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], st["n_free"], **kw)
    p, args, word = _run(st, **kw, in_place=in_place)
    _check(p, word, want, faults)
    if not in_place:   # the state is as it was: the same plan again gives the same
        word.zero_()
        abi.lora_kv4_plan(p, *args, depths=None if depths is None else _i32(depths), dev_status=word)
        _check(p, word, want, faults)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,q_max", [(3, 9), (256, 90), (257, 5), (700, 60), (1024, 3), (1027, 4), (1100, 50), (4095, 5)])
def test_arrays_off_16_bytes(n, q_max, in_place):
    """Lengths and tables that start four bytes behind a 16-byte boundary, at each count of sequences and rows to a thread."""
    rng = np.random.default_rng(n)
    st = _state(rng, n, 32, 300, 3 * n, q_max=q_max)
    rows = int(np.maximum(st["q"], 0).sum()) + n % 5
    want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], st["n_free"], page=32, max_rows=rows, max_q=q_max, max_ctx=300)
    off = lambda a: _i32(np.concatenate([[-9], a]))[1:]
    more = {} if in_place else dict(n_free_out=off([-5]), held_out=off(np.full(n, -5)))
    p = store.KV4Plan(off(st["free"]), off([st["n_free"]]), off(st["held"]), _i32(st["table"]), page_size=32, max_rows=rows, max_q_len=q_max,
                      max_ctx_len=300, **more)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_kv4_plan(p, off(st["q"]), off(st["lens"]), dev_status=word)
    _check(p, word, want, faults)


@pytest.mark.parametrize("n,spare", [(8, 0), (8, 3), (300, 20), (4096, 100)])
def test_too_few_pages(n, spare):
    rng = np.random.default_rng(spare + n)
    st = _state(rng, n, 16, 100, spare, ended=0.02, extra=0)
    kw = dict(page=16, max_rows=int(np.maximum(st["q"], 0).sum()), max_q=4, max_ctx=100)
    want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], st["n_free"], **kw)
    p, _, word = _run(st, **kw, in_place=True)
    _check(p, word, want, faults)
    if (n, spare) != (8, 3):   # three pages are enough there
        assert faults & abi.LORA_DEV_NO_PAGES


def test_faults():
    """Inconsistent lengths and counters: such sequences have no place, and nothing is read or written out of range."""
    rng = np.random.default_rng(5)
    st = _state(rng, 40, 16, 100, 60, ended=0.0, idle=0.0)
    top = np.int64(2 ** 31 - 1)
    for s, k, v in ((3, "q", 5), (5, "q", top), (7, "lens", -1), (9, "lens", 100), (11, "lens", top), (13, "held", -1), (15, "held", 8),
                    (17, "held", top), (19, "lens", -top)):
        st[k][s] = v
    st["q"][21], st["held"][21] = -1, 8
    st["q"][23], st["held"][23] = -int(top), -3
    for rows in (60, 3, 0, 500):
        kw = dict(page=16, max_rows=rows, max_q=4, max_ctx=100)
        want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], st["n_free"], **kw)
        assert faults & abi.LORA_DEV_BAD_SEGMENT
        _check(*[r for i, r in enumerate(_run(st, **kw)) if i != 1], want, faults)
    for n_free in (-1, len(st["free"]) + 1, int(top)):
        want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], n_free, **kw)
        assert faults & abi.LORA_DEV_BAD_PAGE
        p, _, word = _run({**st, "n_free": n_free}, **kw)
        _check(p, word, want, faults)


def test_pages_given_back_past_the_last():
    st = _state(np.random.default_rng(6), 20, 16, 64, 3, ended=1.0)
    st["n_free"] = len(st["free"]) - 2
    kw = dict(page=16, max_rows=0, max_q=1, max_ctx=64)
    want, faults = R.plan(st["q"], st["lens"], st["held"], st["table"], st["free"], st["n_free"], **kw)
    assert faults == abi.LORA_DEV_BAD_PAGE
    p, _, word = _run(st, **kw)
    _check(p, word, want, faults)


def test_no_sequences():
    p = store.KV4Plan.empty(0, 9, 16, max_rows=5, max_q_len=1, max_ctx_len=64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    p.row_seq.fill_(3)
    abi.lora_kv4_plan(p, none, none)
    assert p.q_starts.tolist() == [0] and p.row_seq.tolist() == [-1] * 5 and int(p.n_free_out) == 9


def test_stream_and_replay():
    """Steps of a captured plan on a side stream: requests grow, end and come in, the tables refilled in place."""
    rng = np.random.default_rng(8)
    n, page, max_ctx, rows = 12, 16, 120, 60
    side = torch.cuda.Stream()
    p = store.KV4Plan.empty(n, 70, page, max_rows=rows, max_q_len=9, max_ctx_len=max_ctx)
    q, lens = _i32(np.zeros(n)), _i32(np.zeros(n))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        abi.lora_kv4_plan(p, q, lens, dev_status=word)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        abi.lora_kv4_plan(p, q, lens, dev_status=word)
    st = dict(lens=np.zeros(n, np.int64), held=np.zeros(n, np.int64), table=p.block_table.cpu().numpy().astype(np.int64),
              free=p.free_pages.cpu().numpy().astype(np.int64), n_free=70)
    for step in range(40):
        ql = np.where(st["lens"] == 0, rng.integers(0, 10, n), np.where(rng.random(n) < 0.1, -1, rng.integers(0, 6, n)))
        ql[np.cumsum(np.maximum(ql, 0)) > rows] = 0
        want, faults = R.plan(ql, st["lens"], st["held"], st["table"], st["free"], st["n_free"], page=page, max_rows=rows, max_q=9, max_ctx=max_ctx)
        q.copy_(_i32(ql))
        lens.copy_(_i32(st["lens"]))
        word.zero_()
        g.replay()
        torch.cuda.synchronize()
        _check(p, word, want, faults)
        kept = np.where(ql < 0, 0, np.where(want["ctx_lens"] > 0, want["ctx_lens"] - rng.integers(0, 3, n) * (ql > 2), st["lens"]))
        st = dict(lens=kept, held=want["held"], table=want["block_table"], free=want["free_pages"], n_free=want["n_free"])
