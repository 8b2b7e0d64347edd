"""The host helpers of the binding work where torch cannot be imported."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import sys
sys.modules["torch"] = None            # importing it raises ImportError
import numpy as np
from lora_serving_gb300 import abi, build
build()
assert abi.lora_slot_rank([3, 9]) == 16
m = abi.lora_build_metadata(np.array([0, 0, 1, -1, 1], np.int32), 2, 2)
assert m["n_segs"] >= 1 and sorted(m["perm"]) == sorted(set(m["perm"]))
a, b = abi.lora_prepare_adapter(np.zeros((3, 8), np.uint16), np.zeros((16, 3), np.uint16), 2.0, False, 8)
assert a.shape == (8, 8) and b.shape == (16, 8)
assert abi.lora_kv4_block_bytes(64, 128) == 64 * 144
try:
    abi.lora_rms_norm(None, None, 1e-5)
except RuntimeError as e:
    assert "torch" in str(e)
else:
    raise AssertionError
print("done")
"""


def test_host_helpers_without_torch():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr
