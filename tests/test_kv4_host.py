"""Host-side checks of the norm's and the 4-bit cache's entry points: sizes,
and refusals before anything is enqueued (no kernel launches here)."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from lora_serving_gb300 import abi, build, store

P = 1 << 20          # an aligned address that no refused call dereferences


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return abi.load()


def _status(code):
    return abi.STATUS[code]


def test_block_bytes():
    assert abi.lora_kv4_block_bytes(64, 128) == 64 * (128 + 16)
    assert abi.lora_kv4_block_bytes(16, 64) == 16 * (64 + 8)
    for page, dim in ((8, 128), (48, 128), (512, 64), (64, 96), (64, 256), (0, 64), (-16, 64)):
        assert abi.lora_kv4_block_bytes(page, dim) == 0


def test_workspace_bytes():
    f = abi.lora_kv4_attend_workspace_bytes
    assert f(32, 8, 128, 1) > 0 and f(64, 1, 64, 2048) > 0
    for bad in ((0, 8, 128, 1), (32, 0, 128, 1), (32, 8, 96, 1), (33, 8, 128, 1), (65, 1, 128, 1), (8, 8, 64, -1)):
        assert f(*bad) == 0


NORM = dict(y=P, ld_y=64, y8=P, ld_y8=64, scales=P, ld_scales=1, group=0, ro=P, ld_ro=64, x=P, ld_x=64, r=P, ld_r=64,
            w=P, n=4, width=64, eps=1e-5, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), "INVALID_ARG"), (dict(w=0), "INVALID_ARG"), (dict(y=0, y8=0), "INVALID_ARG"),
    (dict(scales=0), "INVALID_ARG"), (dict(ro=0), "INVALID_ARG"), (dict(r=0), "INVALID_ARG"),
    (dict(n=-1), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(group=64), "SHAPE"), (dict(group=-128), "SHAPE"), (dict(width=65544, ld_x=65544), "SHAPE"),
    (dict(ld_x=56), "SHAPE"), (dict(ld_y=56), "SHAPE"), (dict(ld_y8=56), "SHAPE"), (dict(ld_r=56), "SHAPE"),
    (dict(ld_ro=56), "SHAPE"), (dict(ld_scales=0), "SHAPE"),
    (dict(width=136, group=128, ld_scales=1, ld_x=136, ld_y=136, ld_y8=136, ld_r=136, ld_ro=136), "SHAPE"),
    (dict(width=60), "ALIGNMENT"), (dict(x=P + 8), "ALIGNMENT"), (dict(ld_x=68), "ALIGNMENT"),
    (dict(y=P + 2), "ALIGNMENT"), (dict(w=P + 2), "ALIGNMENT"), (dict(y8=P + 4), "ALIGNMENT"),
    (dict(ld_y8=65), "ALIGNMENT"), (dict(scales=P + 2), "ALIGNMENT"), (dict(r=P + 4), "ALIGNMENT"),
])
def test_norm_refusals(_lib, change, want):
    assert _status(_lib.lora_rms_norm(*{**NORM, **change}.values())) == "LORA_ERR_" + want


def _cache(**k):
    v = dict(pages=P, page_stride=2 * 64 * 144, n_pages=4, page_size=64, n_kv=2, head_dim=128) | k
    return abi.lora_kv4_cache_t(*v.values())


def _batch(**k):
    v = dict(q_starts=P, ctx_lens=P, block_table=P, ld_table=2, n_seqs=3, n_rows=5, max_q_len=3, max_ctx_len=128) | k
    return abi.lora_kv4_batch_t(*v.values())


BAD_CACHES = [(dict(pages=0), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(n_kv=0), "INVALID_ARG"),
              (dict(page_size=48), "SHAPE"), (dict(page_size=8), "SHAPE"), (dict(head_dim=96), "SHAPE"),
              (dict(page_stride=2 * 64 * 144 - 16), "SHAPE"), (dict(page_stride=2 * 64 * 144 + 8), "ALIGNMENT"),
              (dict(pages=P + 8), "ALIGNMENT"), (dict(n_kv=3), "SHAPE")]
BAD_BATCHES = [(dict(q_starts=0), "INVALID_ARG"), (dict(ctx_lens=0), "INVALID_ARG"), (dict(block_table=0), "INVALID_ARG"),
               (dict(n_seqs=-1), "INVALID_ARG"), (dict(n_rows=-1), "INVALID_ARG"), (dict(max_q_len=-1), "INVALID_ARG"),
               (dict(max_ctx_len=-1), "INVALID_ARG"), (dict(n_seqs=0), "METADATA"), (dict(ld_table=1), "SHAPE"),
               (dict(max_ctx_len=129), "SHAPE"), (dict(q_starts=P + 2), "ALIGNMENT")]

APPEND = dict(q=P, ld_q=512, x=P, ld_x=1024, n_heads=4, q_off=0, k_off=512, v_off=768, rope=P, rot=128, max_pos=100,
              pos=P, ld_pos=3, pairs=(24, 20, 20), axes=3, cache={}, batch={}, st=0, stream=0)


def _append(lib, change):
    v = {**APPEND, **change}
    c, b = _cache(**v["cache"]), _batch(**v["batch"])
    v["cache"], v["batch"] = ctypes.byref(c), ctypes.byref(b)
    v["pairs"] = (ctypes.c_int * 4)(*v["pairs"]) if v["pairs"] is not None else None
    return _status(lib.lora_kv4_append(*v.values()))


@pytest.mark.parametrize("change,want", [
    (dict(q=0), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(n_heads=0), "INVALID_ARG"), (dict(q_off=-8), "INVALID_ARG"),
    (dict(rope=0), "INVALID_ARG"), (dict(max_pos=0), "INVALID_ARG"), (dict(pairs=None), "INVALID_ARG"),
    (dict(axes=0), "INVALID_ARG"), (dict(axes=4), "INVALID_ARG"), (dict(pairs=(84, -20, 0)), "INVALID_ARG"),
    (dict(rot=-16), "INVALID_ARG"),
    (dict(ld_q=504), "SHAPE"), (dict(v_off=776), "SHAPE"), (dict(k_off=504), "SHAPE"), (dict(v_off=512), "SHAPE"),
    (dict(q_off=512, k_off=0, v_off=256, n_heads=5), "SHAPE"), (dict(rot=144, pairs=(72, 0, 0)), "SHAPE"),
    (dict(pairs=(24, 20, 19)), "SHAPE"), (dict(axes=2), "SHAPE"), (dict(ld_pos=2), "SHAPE"),
    (dict(n_heads=1000), "SHAPE"),
    (dict(rot=120, pairs=(20, 20, 20)), "ALIGNMENT"), (dict(q=P + 8), "ALIGNMENT"), (dict(rope=P + 4), "ALIGNMENT"),
    (dict(pos=P + 1), "ALIGNMENT"), (dict(k_off=516, v_off=772, ld_x=1032), "ALIGNMENT"),
] + [(dict(cache=c), w) for c, w in BAD_CACHES if "n_kv" not in c] + [(dict(batch=b), w) for b, w in BAD_BATCHES])
def test_append_refusals(_lib, change, want):
    assert _append(_lib, change) == "LORA_ERR_" + want


def test_empty_batches_are_no_ops(_lib):
    assert _append(_lib, dict(batch=dict(n_rows=0, n_seqs=0, q_starts=0))) == "LORA_OK"
    c, b = _cache(), _batch(n_rows=0)
    assert _lib.lora_kv4_read(0, 0, 0, 0, ctypes.byref(c), ctypes.byref(b), 0, 0) == 0
    assert _lib.lora_kv4_attend(0, 0, 0, 0, 4, 0.1, 0, ctypes.byref(c), ctypes.byref(b), 0, 0, 0, 0) == 0
    assert _lib.lora_rms_norm(*{**NORM, "n": 0}.values()) == 0


@pytest.mark.parametrize("change,want", [
    (dict(k=0), "INVALID_ARG"), (dict(v=0), "INVALID_ARG"), (dict(ld_k=248), "SHAPE"), (dict(ld_v=260), "ALIGNMENT"),
    (dict(k=P + 2), "ALIGNMENT"),
] + [(dict(cache=c), w) for c, w in BAD_CACHES] + [(dict(batch=b), w) for b, w in BAD_BATCHES])
def test_read_refusals(_lib, change, want):
    v = {**dict(k=P, ld_k=256, v=P, ld_v=256, cache={}, batch={}, st=0, stream=0), **change}
    c, b = _cache(**v["cache"]), _batch(**v["batch"])
    v["cache"], v["batch"] = ctypes.byref(c), ctypes.byref(b)
    assert _status(_lib.lora_kv4_read(*v.values())) == "LORA_ERR_" + want


@pytest.mark.parametrize("change,want", [
    (dict(out=0), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"), (dict(n_heads=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(n_heads=5), "SHAPE"), (dict(n_heads=130, ld_q=1 << 15, ld_out=1 << 15), "SHAPE"), (dict(ld_q=504), "SHAPE"),
    (dict(ld_out=504), "SHAPE"), (dict(out=P + 8), "ALIGNMENT"), (dict(ld_q=516), "ALIGNMENT"),
    (dict(ws=0), "WORKSPACE"), (dict(ws_bytes=0), "WORKSPACE"), (dict(ws=P + 128), "ALIGNMENT"),
] + [(dict(cache=c), w) for c, w in BAD_CACHES] + [(dict(batch=b), w) for b, w in BAD_BATCHES])
def test_attend_refusals(_lib, change, want):
    v = {**dict(out=P, ld_out=512, q=P, ld_q=512, n_heads=4, scale=0.1, window=0, cache={}, batch={}, ws=P,
                ws_bytes=1 << 30, st=0, stream=0), **change}
    c, b = _cache(**v["cache"]), _batch(**v["batch"])
    v["cache"], v["batch"] = ctypes.byref(c), ctypes.byref(b)
    assert _status(_lib.lora_kv4_attend(*v.values())) == "LORA_ERR_" + want


@pytest.mark.parametrize("batch,want", [
    (dict(n_rows=1 << 24, max_q_len=1 << 24, max_ctx_len=1 << 24, n_seqs=1), "SHAPE"),      # 2^17 blocks of 2^17 tiles
    (dict(n_rows=4096, max_q_len=1, max_ctx_len=1 << 24, n_seqs=4096), "SHAPE"),            # 2^13 units of 2^19 tiles
    (dict(n_rows=4096, max_q_len=1, max_ctx_len=1 << 22, n_seqs=4096), "WORKSPACE"),        # 2^30: counted in 32 bits
])
def test_attend_refuses_more_tiles_than_31_bits(_lib, batch, want):
    c, b = _cache(), _batch(**batch, ld_table=1 << 20)
    args = [P, 512, P, 512, 4, 0.1, 0, ctypes.byref(c), ctypes.byref(b), 0, 0, 0, 0]
    assert _status(_lib.lora_kv4_attend(*args)) == "LORA_ERR_" + want
    args[6] = 4096                                                                          # a window bounds the tiles
    assert _status(_lib.lora_kv4_attend(*args)) == "LORA_ERR_WORKSPACE"


def test_null_structs(_lib):
    c, b = _cache(), _batch()
    assert _status(_lib.lora_kv4_read(P, 256, P, 256, None, ctypes.byref(b), 0, 0)) == "LORA_ERR_INVALID_ARG"
    assert _status(_lib.lora_kv4_read(P, 256, P, 256, ctypes.byref(c), None, 0, 0)) == "LORA_ERR_INVALID_ARG"


def test_python_handles_refuse_host_memory_and_wrong_shapes():
    with pytest.raises(ValueError):
        store.KV4Cache(2, 64, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        store.KV4Cache(2, 48, 2, 128, device="cpu")
    z = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        store.KV4Batch(z, z, z.view(3, 1), n_rows=1, max_q_len=1, max_ctx_len=1)


@pytest.mark.parametrize("call", ["norm", "append", "read", "attend"])
def test_python_calls_refuse_host_tensors(_lib, call):
    """A host pointer handed to a kernel is an illegal address."""
    c, b = _cache(), _batch()
    cache, batch = SimpleNamespace(addr=ctypes.addressof(c)), SimpleNamespace(addr=ctypes.addressof(b))
    x = torch.zeros(5, 1024, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        if call == "norm":
            abi.lora_rms_norm(x, torch.ones(1024, dtype=torch.bfloat16), 1e-5, y=x)
        elif call == "append":
            abi.lora_kv4_append(x, x, cache, batch, n_heads=4, q_off=0, k_off=512, v_off=768)
        elif call == "read":
            abi.lora_kv4_read(x, x, cache, batch)
        else:
            abi.lora_kv4_attend(x, x, cache, batch, x, n_heads=4, scale=0.1)


def test_python_calls_refuse_what_is_no_tensor(_lib):
    c, b = _cache(), _batch()
    cache, batch = SimpleNamespace(addr=ctypes.addressof(c)), SimpleNamespace(addr=ctypes.addressof(b))
    with pytest.raises(AttributeError):
        abi.lora_kv4_read([1.0], [1.0], cache, batch)
    with pytest.raises(ValueError, match="no cache"):
        abi.lora_kv4_read(None, None, SimpleNamespace(addr=0), batch)
    with pytest.raises(ValueError, match="out of range"):
        abi.lora_kv4_attend(None, None, cache, batch, None, n_heads=1 << 40, scale=0.1)
    with pytest.raises(TypeError):
        abi.lora_kv4_attend(None, None, cache, batch, None, n_heads=4, scale="a")
    for bad in (torch.ones(8), torch.ones(16)[::2], torch.ones(8, 2)):   # a weight that is not the row's
        with pytest.raises(ValueError, match="adjacent"):
            abi.lora_rms_norm(torch.zeros(2, 16), bad, 1e-5)
    with pytest.raises(ValueError, match="2-D"):
        abi.lora_rms_norm(torch.zeros(16), torch.ones(16), 1e-5)
