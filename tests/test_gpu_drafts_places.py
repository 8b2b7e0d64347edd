"""Sequences that a plan gives no place in the batch: what append, attention and keep then do with them."""
import numpy as np
import pytest
import torch

from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu

PAGE, H, KV, D, MAX_Q, MAX_ROWS, MAX_CTX = 16, 4, 2, 64, 6, 10, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


SEQS = [  # rows, cached positions, pages, rows kept, cached positions afterwards
    (4, 20, 2, 2, 22),
    (-1, 10, 1, 0, 0),      # ended
    (4, 5, 1, 1, 6),
    (4, 30, 2, 0, 30),      # its rows go past max_rows, two of them inside
    (3, 17, 2, 0, 17),      # all of its rows past max_rows
    (0, 33, 5, 0, 33),      # idle, with more pages than a row of the table has
    (0, 40, 3, 0, 40),      # idle
    (0, 0, 0, 0, 0),        # idle, nothing cached
    (9, 12, 1, 0, 12),      # more than max_q_len rows, all past max_rows
]


@pytest.mark.parametrize("in_place", [False, True])
def test_a_sequence_without_a_place_keeps_its_length(in_place):
    q, cached, held, kept, after = (list(a) for a in zip(*SEQS))
    n, wide = len(q), MAX_CTX // PAGE
    table = np.full((n, wide), -1)
    at = 0
    for s, h in enumerate(held):
        table[s, :min(h, wide)] = np.arange(at, at + min(h, wide))
        at += min(h, wide)
    free = np.concatenate([np.arange(at, at + 4), np.full(at, -1)])
    more = {} if in_place else dict(n_free_out=_i32([-5]), held_out=_i32([-5] * n))
    p = store.KV4Plan(_i32(free), _i32([4]), _i32(held), _i32(table), page_size=PAGE, max_rows=MAX_ROWS, max_q_len=MAX_Q, max_ctx_len=MAX_CTX, **more)
    cache = store.KV4Cache(len(free), PAGE, KV, D)
    lens, st = _i32(cached), _i32([0])
    abi.lora_kv4_plan(p, _i32(q), lens, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    assert p.q_starts.tolist() == [0, 4, 4, 8, 10, 10, 10, 10, 10, 10] and p.ctx_lens.tolist() == [24, 0, 9, 0, 0, 0, 40, 0, 0]
    st.zero_()
    qkv = torch.randn(MAX_ROWS, (H + 2 * KV) * D, device="cuda").bfloat16()
    qr, o = (torch.full((MAX_ROWS, H * D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    abi.lora_kv4_append(qr, qkv, cache, p.batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, dev_status=st)
    tree = torch.full((MAX_ROWS, 1), -1, dtype=torch.int32, device="cuda")
    abi.lora_kv4_attend_tree(o, qr, cache, p.batch, tree, store.kv4_workspace(cache, H, p.batch), n_heads=H, scale=0.1, dev_status=st)
    assert (o[8:] == 0).all() and (qr[8:] == 7).all()
    path = _i32([[0, 1]] * n)
    abi.lora_kv4_keep(store.KV4Layers([cache]), p.batch, _i32(kept), path, lens=lens, dev_status=st)
    assert lens.tolist() == after and abi.lora_read_device_status(st) == 0
    # the next step goes on behind them
    if in_place:
        abi.lora_kv4_plan(p, _i32([0, -1, 0, 1, 1, 0, 0, 0, 1]), lens, dev_status=st)
        assert p.ctx_lens.tolist() == [22, 0, 6, 31, 18, 0, 40, 0, 13]


def test_more_rows_than_the_bound():
    """A sequence past max_q_len has no place either, but its rows stay in the batch, whose bound they pass: append,
    attention and keep skip it, flagged, and its rows are not written (no zeros)."""
    q, cached = [9, 2, 3], [12, 20, 0]
    p = store.KV4Plan.empty(3, 8, PAGE, max_rows=20, max_q_len=MAX_Q, max_ctx_len=MAX_CTX)
    p.held.copy_(_i32([1, 2, 0]))
    p.block_table[:, :2] = _i32([[0, -1], [1, 2], [-1, -1]])
    p.n_free.fill_(5)
    cache, lens, st = store.KV4Cache(8, PAGE, KV, D), _i32(cached), _i32([0])
    abi.lora_kv4_plan(p, _i32(q), lens, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    assert p.q_starts.tolist() == [0, 9, 11, 14] and p.ctx_lens.tolist() == [0, 22, 3]
    assert p.row_seq.tolist() == [-1] * 9 + [1, 1, 2, 2, 2] + [-1] * 6
    qkv = torch.randn(20, (H + 2 * KV) * D, device="cuda").bfloat16()
    qr, o = (torch.full((20, H * D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tree, ws = torch.full((20, 1), -1, dtype=torch.int32, device="cuda"), store.kv4_workspace(cache, H, p.batch)
    for call in (lambda: abi.lora_kv4_append(qr, qkv, cache, p.batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, dev_status=st),
                 lambda: abi.lora_kv4_attend_tree(o, qr, cache, p.batch, tree, ws, n_heads=H, scale=0.1, dev_status=st),
                 lambda: abi.lora_kv4_keep(store.KV4Layers([cache]), p.batch, _i32([2, 1, 1]), _i32([[0, 1]] * 3), lens=lens, dev_status=st)):
        st.zero_()
        call()
        assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    for t in (qr, o):
        assert (t[:9] == 7).all() and (t[14:] == 7).all() and not (t[9:14] == 7).all(1).any()
    assert lens.tolist() == [12, 21, 1]
