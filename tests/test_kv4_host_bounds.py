"""Batches whose positions or rows the attention kernels could not count in 32
bits are refused on the host."""
import ctypes

import pytest

from lora_serving_gb300 import abi, build

P = 1 << 20          # an aligned address that no refused call dereferences


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return abi.load()


def _attend(lib, window=0, n_heads=4, **batch):
    """Without a workspace: what passes the checks of its shape ends there."""
    c = abi.lora_kv4_cache_t(pages=P, page_stride=256 * 72, n_pages=4, page_size=256, n_kv=1, head_dim=64)
    v = dict(q_starts=P, ctx_lens=P, block_table=P, ld_table=1 << 23, n_seqs=1, n_rows=1, max_q_len=1, max_ctx_len=128) | batch
    b = abi.lora_kv4_batch_t(*v.values())
    return abi.STATUS[lib.lora_kv4_attend(P, 64 * n_heads, P, 64 * n_heads, n_heads, 0.1, window, ctypes.byref(c), ctypes.byref(b), 0, 0, 0, 0)]


@pytest.mark.parametrize("window", [0, 4096, 2 ** 31 - 1])
@pytest.mark.parametrize("ctx,ok", [(2 ** 30, True), (2 ** 30 + 1, False), (2 ** 31 - 40, False), (2 ** 31 - 1, False)])
def test_positions(_lib, ctx, ok, window):
    assert _attend(_lib, window, max_ctx_len=ctx) == ("LORA_ERR_WORKSPACE" if ok else "LORA_ERR_SHAPE")


@pytest.mark.parametrize("rows,heads,ok", [(2 ** 24, 64, True), (2 ** 24 + 1, 64, False), (2 ** 30, 1, True), (2 ** 31 - 1, 1, False), (2 ** 28, 64, False)])
def test_rows(_lib, rows, heads, ok):
    assert _attend(_lib, n_heads=heads, n_rows=rows, max_q_len=rows) == ("LORA_ERR_WORKSPACE" if ok else "LORA_ERR_SHAPE")
    # the bound is of the rows there are, not of how long a sequence might be
    assert _attend(_lib, n_heads=heads, n_rows=3, max_q_len=rows) == "LORA_ERR_WORKSPACE"
