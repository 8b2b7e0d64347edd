"""What does not need the C extension does not fail for want of it."""
import importlib
import os

import pytest

import lora_serving_gb300
from lora_serving_gb300 import abi


def test_the_library_without_the_extension(monkeypatch, tmp_path):
    lora_serving_gb300.build()
    mod = importlib.import_module("lora_serving_gb300.build")
    calls = str(tmp_path / "_pycalls.so")
    monkeypatch.setattr(mod, "CALLS", calls)
    for cc in ("false", "/no/such/compiler"):
        monkeypatch.setenv("CC", cc)
        with open(calls, "w"):                                     # an older one goes
            os.utime(calls, (0, 0))
        with pytest.warns(UserWarning, match="cannot be called from Python"):
            assert lora_serving_gb300.build() == mod.LIB
    assert os.path.exists(mod.LIB) and not os.path.exists(calls) and os.listdir(tmp_path) == []
    assert abi.lora_slot_rank([3, 9]) > 0
    monkeypatch.setattr(abi, "CALLS_PATH", calls)
    with pytest.raises(RuntimeError, match="is missing"):
        abi._load_calls()
    monkeypatch.delenv("CC")
    lora_serving_gb300.build()
    assert os.path.exists(calls)
