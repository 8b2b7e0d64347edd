"""lora_kv4_append from Python: the columns of x that the call reads lie inside
x, not only inside the buffer that x is a slice of.  (A stand-in for a CUDA
tensor: what is refused is refused before its address is used.)"""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from lora_serving_gb300 import abi, build

P = 1 << 20
H, KV, D, T = 4, 2, 128, 5
W = (H + 2 * KV) * D


class Fake:
    is_cuda = True
    device = "cuda:0"
    dtype = torch.bfloat16

    def __init__(self, rows, cols, ld):
        self.shape, self._ld = (rows, cols), ld

    def stride(self):
        return (self._ld, 1)

    def data_ptr(self):
        return P


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return abi.load()


@pytest.mark.parametrize("cols,off", [(W - 8, (0, H * D, (H + KV) * D)),          # v's last columns
                                      (W, (8, H * D + 8, (H + KV) * D + 8)), (W, (KV * D + 8, 0, KV * D + H * D + 8)),
                                      (H * D, (0, H * D, (H + KV) * D)), (0, (0, H * D, (H + KV) * D)),
                                      (W, (2 ** 31 - 8, 0, KV * D)), (W, (2 * KV * D, 2 ** 31 - 8, 0)), (W, (2 * KV * D, 0, 2 ** 31 - 8))])
def test_append_refuses_columns_past_x(cols, off):
    c = abi.lora_kv4_cache_t(pages=P, page_stride=2 * 64 * 144, n_pages=4, page_size=64, n_kv=KV, head_dim=D)
    b = abi.lora_kv4_batch_t(q_starts=P, ctx_lens=P, block_table=P, ld_table=2, n_seqs=3, n_rows=T, max_q_len=3, max_ctx_len=128)
    cache, batch = SimpleNamespace(addr=ctypes.addressof(c)), SimpleNamespace(addr=ctypes.addressof(b))
    with pytest.raises(ValueError, match="x must be 2-D with 5 rows"):
        abi.lora_kv4_append(Fake(T, H * D, H * D), Fake(T, cols, 1 << 20), cache, batch, n_heads=H, q_off=off[0], k_off=off[1],
                            v_off=off[2], stream=0)
