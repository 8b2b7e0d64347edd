"""The structs that Python hands to the library, member by member, against the
C sources that read them: names, order and types."""
import ctypes
import os
import re

import pytest

from lora_serving_gb300 import abi

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir)
SCALARS = {"int": ctypes.c_int, "int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "uint64_t": ctypes.c_uint64, "size_t": ctypes.c_size_t,
           "float": ctypes.c_float}


def _members(path, name):
    """[(member, type)] of a typedef struct; pointers of any kind are void*, other structs their names."""
    with open(os.path.join(ROOT, path)) as f:
        text = re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
    out = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = re.match(r"(?:const )?(\w+)\s*(.*)", line, re.S).groups()
        for one in names.split(","):
            stars, member = re.match(r"\s*(\**)\s*(\w+)$", one).groups()
            out.append((member, ctypes.c_void_p if stars else SCALARS.get(kind, kind)))
    return out


def _fields(struct):
    return [(n, t.__name__ if issubclass(t, ctypes.Structure) else t) for n, t in struct._fields_]


@pytest.mark.parametrize("path,name,struct", [
    ("include/lora.h", n, getattr(abi, n)) for n in ("lora_meta_t", "lora_kv4_cache_t", "lora_kv4_batch_t", "lora_kv4_pool_t", "lora_logits_rules_t")
] + [("lora_serving_gb300/csrc/pycalls.c", "plan_t", abi.plan_args_t)], ids=lambda v: v if isinstance(v, str) else "")
def test_members(path, name, struct):
    assert _fields(struct) == _members(path, name)


def test_what_the_comparison_would_show():
    """Two members of one type that change places, and a member that is missing."""
    want = _members("include/lora.h", "lora_kv4_pool_t")
    held, out = [m for m, _ in want].index("held"), [m for m, _ in want].index("held_out")
    want[held], want[out] = want[out], want[held]
    assert _fields(abi.lora_kv4_pool_t) != want and sorted(_fields(abi.lora_kv4_pool_t), key=str) == sorted(want, key=str)
    assert _fields(abi.lora_logits_rules_t)[:-1] != _members("include/lora.h", "lora_logits_rules_t")
