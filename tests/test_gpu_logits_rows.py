"""lora_logits_adjust: entries of its tables that name rows or requests which are not there."""
import numpy as np
import pytest
import torch

from lora_serving_gb300 import abi
from test_gpu_logits import BF, _args, _built, _case, _i32  # noqa: F401

pytestmark = pytest.mark.gpu

TOP, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("first,end", [(TOP, LOW), (5, LOW), (5, LOW + 4), (TOP, -2), (4, 2), (2, LOW), (TOP, TOP)])
def test_row_starts_that_fall(first, end):
    """A request whose rows end before they begin has none: the difference of the two may pass 32 bits.  (Requests 0 and 2 share
    an entry with it, request 3 is as it was.)"""
    V = 3000
    c = _case(5, [2, 2, 2, 2], V, [30] * 4, 6, True, True)
    rules, kw = _args(c)
    x, want = c["x"][:, :V], torch.full((8, V), 7.0, dtype=BF, device="cuda")
    abi.lora_logits_adjust(want, x, rules, **kw)
    starts = [0, first, end, 6, 8]
    out, st = torch.full_like(want, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_logits_adjust(out, x, rules, dev_status=st, **{**kw, "q_starts": _i32(starts)})
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    for t, s in enumerate(np.repeat(np.arange(4), 2)):
        inside = 0 <= starts[s] <= t < starts[s + 1] <= 8
        assert inside if s == 3 else True
        if not inside:
            assert (out[t] == 7).all(), t
    assert torch.equal(out[6:], want[6:])
