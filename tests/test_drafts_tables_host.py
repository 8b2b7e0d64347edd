"""Host-side checks of the tables that drafted decoding's calls share (no kernel launches here)."""
import ctypes

import pytest

from lora_serving_gb300 import abi, build
from test_drafts_host import KEEP, P, _batch, _cache, _status


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    return abi.load()


def test_keep_refuses_misaligned_held_pages(_lib):
    c, b = _cache(), _batch()
    b.held = P + 2
    v = {**KEEP, "caches": ctypes.byref(c), "n": 1, "batch": ctypes.byref(b)}
    assert _status(_lib.lora_kv4_keep(*v.values())) == "LORA_ERR_ALIGNMENT"
