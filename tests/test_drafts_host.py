"""Host-side checks of drafted decoding's entry points: refusals before
anything is enqueued (no kernel launches here)."""
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


def _pool(**k):
    v = dict(free_pages=P, n_free=P, held=P, n_free_out=P, held_out=P, block_table=P, ld_table=4, n_pages=9, page_size=16) | k
    return abi.lora_kv4_pool_t(*v.values())


PLAN = dict(q_starts=P, ctx_lens=P, row_seq=P, positions=P, slots=P, q_lens=P, lens=P + 64, depths=0, n_seqs=3, max_rows=8, max_q=4, max_ctx=64,
            pool={}, st=0, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(q_starts=0), "INVALID_ARG"), (dict(ctx_lens=0), "INVALID_ARG"), (dict(q_lens=0), "INVALID_ARG"), (dict(lens=0), "INVALID_ARG"),
    (dict(lens=P), "INVALID_ARG"), (dict(n_seqs=-1), "INVALID_ARG"), (dict(max_rows=-1), "INVALID_ARG"), (dict(max_q=-1), "INVALID_ARG"),
    (dict(max_ctx=-1), "INVALID_ARG"), (dict(pool=None), "INVALID_ARG"), (dict(pool=dict(n_pages=0)), "INVALID_ARG"),
    (dict(pool=dict(free_pages=0)), "INVALID_ARG"), (dict(pool=dict(n_free=0)), "INVALID_ARG"), (dict(pool=dict(held=0)), "INVALID_ARG"),
    (dict(pool=dict(n_free_out=0)), "INVALID_ARG"), (dict(pool=dict(held_out=0)), "INVALID_ARG"), (dict(pool=dict(block_table=0)), "INVALID_ARG"),
    (dict(pool=dict(page_size=48)), "SHAPE"), (dict(pool=dict(page_size=0)), "SHAPE"), (dict(max_ctx=65), "SHAPE"), (dict(pool=dict(ld_table=3)), "SHAPE"),
    (dict(n_seqs=4097), "SHAPE"), (dict(max_rows=(1 << 30) + 1), "SHAPE"), (dict(max_ctx=(1 << 30) + 1, pool=dict(ld_table=1 << 27)), "SHAPE"),
    (dict(pool=dict(n_pages=(1 << 30) + 1)), "SHAPE"),
    (dict(q_starts=P + 2), "ALIGNMENT"), (dict(slots=P + 4), "ALIGNMENT"), (dict(depths=P + 1), "ALIGNMENT"), (dict(positions=P + 2), "ALIGNMENT"),
    (dict(pool=dict(held=P + 2)), "ALIGNMENT"), (dict(pool=dict(block_table=P + 1)), "ALIGNMENT"),
])
def test_plan_refusals(_lib, change, want):
    v = {**PLAN, **change}
    pool = _pool(**v["pool"]) if v["pool"] is not None else None
    v["pool"] = ctypes.byref(pool) if pool else None
    assert _status(_lib.lora_kv4_plan(*v.values())) == "LORA_ERR_" + want


def _cache(**k):
    v = dict(pages=P, page_stride=2 * 64 * 144, n_pages=4, page_size=64, n_kv=2, head_dim=128) | k
    return abi.lora_kv4_cache_t(*v.values())


def _batch(**k):
    v = dict(q_starts=P, ctx_lens=P, block_table=P, ld_table=2, n_seqs=3, n_rows=5, max_q_len=33, max_ctx_len=128) | k
    return abi.lora_kv4_batch_t(*v.values())


@pytest.mark.parametrize("change,want", [
    (dict(tree=0), "INVALID_ARG"), (dict(ld_tree=1), "SHAPE"), (dict(ld_tree=-1), "SHAPE"), (dict(tree=P + 2), "ALIGNMENT"),
    (dict(out=0), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(n_heads=5), "SHAPE"), (dict(ld_q=504), "SHAPE"), (dict(ld_out=516), "ALIGNMENT"), (dict(ws=0), "WORKSPACE"), (dict(ws_bytes=0), "WORKSPACE"),
    (dict(ws=P + 128), "ALIGNMENT"), (dict(cache=dict(page_size=48)), "SHAPE"), (dict(cache=dict(pages=0)), "INVALID_ARG"),
    (dict(batch=dict(n_seqs=0)), "METADATA"), (dict(batch=dict(max_ctx_len=129)), "SHAPE"), (dict(batch=dict(q_starts=0)), "INVALID_ARG"),
    (dict(batch=dict(n_seqs=4097)), "SHAPE"),
    # every block of a tree sees all of it: more tiles than 31 bits count
    (dict(batch=dict(n_rows=1 << 24, max_q_len=1 << 24, max_ctx_len=1 << 24, n_seqs=1, ld_table=1 << 20), ld_tree=1 << 19, window=4096), "SHAPE"),
])
def test_attend_tree_refusals(_lib, change, want):
    v = {**dict(out=P, ld_out=512, q=P, ld_q=512, n_heads=4, scale=0.1, window=0, tree=P, ld_tree=2, cache={}, batch={}, ws=P, ws_bytes=1 << 30,
                st=0, stream=0), **change}
    c, b = _cache(**v["cache"]), _batch(**v["batch"])
    v["cache"], v["batch"] = ctypes.byref(c), ctypes.byref(b)
    assert _status(_lib.lora_kv4_attend_tree(*v.values())) == "LORA_ERR_" + want


KEEP = dict(caches=[{}], n=None, batch={}, n_keep=P, path=P, ld_path=4, lens=P + 64, st=0, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(n=-1), "INVALID_ARG"), (dict(caches=None, n=1), "INVALID_ARG"), (dict(n_keep=0), "INVALID_ARG"), (dict(path=0), "INVALID_ARG"),
    (dict(lens=P), "INVALID_ARG"), (dict(batch=dict(q_starts=0)), "INVALID_ARG"), (dict(batch=dict(ctx_lens=0, n_rows=0)), "INVALID_ARG"),
    (dict(caches=[{}, {}]), "INVALID_ARG"), (dict(caches=[{}, dict(pages=P << 1, n_kv=1)]), "SHAPE"),
    (dict(caches=[{}, dict(pages=P << 1, page_size=32)]), "SHAPE"), (dict(caches=[{}, dict(pages=P << 1, head_dim=64)]), "SHAPE"),
    (dict(caches=[{}, dict(pages=P << 1, page_stride=16)]), "SHAPE"), (dict(caches=[dict(pages=0)]), "INVALID_ARG"),
    (dict(ld_path=-1), "SHAPE"), (dict(batch=dict(max_ctx_len=129)), "SHAPE"), (dict(batch=dict(max_ctx_len=129, n_rows=0)), "SHAPE"),
    (dict(batch=dict(n_seqs=0)), "METADATA"), (dict(n_keep=P + 2), "ALIGNMENT"), (dict(path=P + 1), "ALIGNMENT"), (dict(lens=P + 6), "ALIGNMENT"),
])
def test_keep_refusals(_lib, change, want):
    v = {**KEEP, **change}
    caches = [_cache(**k) for k in v["caches"] or []]
    arr = (abi.lora_kv4_cache_t * max(1, len(caches)))(*caches)
    b = _batch(**v["batch"])
    v["n"] = len(caches) if v["n"] is None else v["n"]
    v["caches"], v["batch"] = ctypes.byref(arr) if v["caches"] is not None else None, ctypes.byref(b)
    assert _status(_lib.lora_kv4_keep(*v.values())) == "LORA_ERR_" + want


def _rules(**k):
    v = dict(tokens=P, prompt=P, length=P, rep=0, freq=0, pres=0, ids=0, bias=0, n_bias=0, ld_tokens=10, ld_bias=0, n_seqs=5) | k
    return abi.lora_logits_rules_t(*v.values())


LOGITS = dict(out=P, out_type=0, ld_out=104, x=P << 1, type=0, ld=104, n=5, vocab=100, rules={}, row_seq=0, drafts=0, tree=0, ld_tree=0, q_starts=0,
              allowed=0, ld_allowed=0, n_allowed=0, allowed_rows=0, st=0, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(out=0), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(vocab=0), "INVALID_ARG"), (dict(type=2), "INVALID_ARG"),
    (dict(out_type=-1), "INVALID_ARG"), (dict(n=6), "INVALID_ARG"), (dict(x=P, out_type=1), "INVALID_ARG"), (dict(x=P, ld=112), "INVALID_ARG"),
    (dict(rules=dict(tokens=0)), "INVALID_ARG"), (dict(rules=dict(prompt=0)), "INVALID_ARG"), (dict(rules=dict(length=0)), "INVALID_ARG"),
    (dict(rules=dict(n_seqs=0)), "INVALID_ARG"), (dict(rules=dict(ld_tokens=-1)), "INVALID_ARG"), (dict(rules=dict(ids=P, ld_bias=3)), "INVALID_ARG"),
    (dict(rules=dict(ids=P, bias=P, ld_bias=3)), "INVALID_ARG"), (dict(drafts=P, tree=P, ld_tree=1), "INVALID_ARG"),
    (dict(drafts=P, q_starts=P, ld_tree=1), "INVALID_ARG"), (dict(rules=None, drafts=P, tree=P, ld_tree=1, q_starts=P), "INVALID_ARG"),
    (dict(allowed=P, ld_allowed=4, n_allowed=4), "INVALID_ARG"), (dict(allowed=P, ld_allowed=4, n_allowed=0, allowed_rows=P), "INVALID_ARG"),
    (dict(ld=96), "SHAPE"), (dict(ld_out=96), "SHAPE"), (dict(vocab=(1 << 25) + 1), "SHAPE"), (dict(allowed=P, ld_allowed=3, n_allowed=5), "SHAPE"),
    (dict(rules=dict(ld_tokens=1 << 20)), "SHAPE"), (dict(rules=dict(ld_tokens=(1 << 20) - 40), drafts=P, tree=P, ld_tree=2, q_starts=P), "SHAPE"),
    (dict(rules=dict(ids=P, bias=P, n_bias=P, ld_bias=2048)), "SHAPE"), (dict(drafts=P, tree=P, ld_tree=0, q_starts=P), "SHAPE"),
    (dict(n=(1 << 30) + 1, rules=None), "SHAPE"), (dict(n=1 << 20, vocab=1 << 25, ld=1 << 25, ld_out=1 << 25, rules=None), "SHAPE"),
    (dict(ld=108), "ALIGNMENT"), (dict(x=P + 8), "ALIGNMENT"), (dict(out=P + 4), "ALIGNMENT"), (dict(row_seq=P + 2), "ALIGNMENT"),
    (dict(rules=dict(rep=P + 1)), "ALIGNMENT"), (dict(allowed=P + 2, ld_allowed=4, n_allowed=5), "ALIGNMENT"),
])
def test_logits_refusals(_lib, change, want):
    v = {**LOGITS, **change}
    r = _rules(**v["rules"]) if v["rules"] is not None else None
    v["rules"] = ctypes.byref(r) if r else None
    assert _status(_lib.lora_logits_adjust(*v.values())) == "LORA_ERR_" + want


def test_empty_calls_are_no_ops(_lib):
    v = {**LOGITS, "n": 0, "rules": None, "out": 0}
    assert _lib.lora_logits_adjust(*v.values()) == 0
    b, c = _batch(n_rows=0), _cache()
    assert _lib.lora_kv4_attend_tree(0, 0, 0, 0, 4, 0.1, 0, 0, 0, ctypes.byref(c), ctypes.byref(b), 0, 0, 0, 0) == 0
    assert _lib.lora_kv4_keep(None, 0, ctypes.byref(b), 0, 0, 0, 0, 0, 0) == 0
    b = _batch(n_rows=0, n_seqs=0)
    assert _lib.lora_kv4_keep(ctypes.byref(c), 1, ctypes.byref(b), 0, 0, 0, 0, 0, 0) == 0
    assert _status(_lib.lora_kv4_keep(ctypes.byref(c), 1, None, P, P, 1, 0, 0, 0)) == "LORA_ERR_INVALID_ARG"
    assert _status(_lib.lora_kv4_attend_tree(P, 8, P, 8, 4, 0.1, 0, P, 1, ctypes.byref(c), None, P, 1, 0, 0)) == "LORA_ERR_INVALID_ARG"


def test_struct_layouts():
    """The Python structs against the header's, member by member."""
    assert ctypes.sizeof(abi.lora_kv4_pool_t) == 6 * 8 + 3 * 4 + 4
    assert ctypes.sizeof(abi.lora_logits_rules_t) == 9 * 8 + 3 * 4 + 4
    assert abi.plan_args_t.pool.offset == 5 * 8 + 4 * 4


def test_python_handles_refuse_host_memory():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        store.KV4Plan(z, z, z, z.view(4, 1), page_size=16, max_rows=4, max_q_len=1, max_ctx_len=16)
    with pytest.raises(ValueError):
        store.KV4Plan(z, z, z, z.view(2, 2), page_size=16, max_rows=4, max_q_len=1, max_ctx_len=16)
    with pytest.raises(ValueError):
        store.LogitsRules(z.view(4, 1), z, z)
    with pytest.raises(ValueError, match="together"):
        store.LogitsRules(z.view(4, 1), z, z, bias_ids=z.view(4, 1))


@pytest.mark.parametrize("call", ["plan", "tree", "keep", "logits"])
def test_python_calls_refuse_host_tensors(_lib, call):
    """A host pointer handed to a kernel is an illegal address."""
    c, b = _cache(), _batch()
    cache, batch = SimpleNamespace(addr=ctypes.addressof(c), n=1), SimpleNamespace(addr=ctypes.addressof(b))
    x, z = torch.zeros(5, 1024, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    plan = abi.plan_args_t(n_seqs=3, max_rows=8)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        if call == "plan":
            abi.lora_kv4_plan(SimpleNamespace(addr=ctypes.addressof(plan)), z, z)
        elif call == "tree":
            abi.lora_kv4_attend_tree(x, x, cache, batch, z.view(8, 1), x, n_heads=4, scale=0.1)
        elif call == "keep":
            abi.lora_kv4_keep(cache, batch, z, z.view(4, 2))
        else:
            abi.lora_logits_adjust(x, x)


def test_python_calls_refuse_what_is_no_handle(_lib):
    none = SimpleNamespace(addr=0, n=0)
    with pytest.raises(ValueError, match="no plan"):
        abi.lora_kv4_plan(none, None, None)
    with pytest.raises(ValueError, match="no cache"):
        abi.lora_kv4_attend_tree(None, None, none, none, None, None, n_heads=1, scale=0.1)
    with pytest.raises(ValueError, match="no cache"):
        abi.lora_kv4_keep(none, none, None, None)
    with pytest.raises(AttributeError):
        abi.lora_logits_adjust([1.0], [1.0])
