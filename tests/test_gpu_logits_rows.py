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


@pytest.mark.parametrize("rows", [8, 700])      # short chunks and long ones
def test_rows_of_no_request_without_rules(rows):
    """-1 is a row that is left; what lies below is refused and left, with rules or without."""
    V = 3000
    x = torch.randn(rows, V, device="cuda").to(BF)
    sets = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, -(-V // 32)), device="cuda").to(torch.int32)
    seq, none = np.zeros(rows), _i32(np.zeros(rows))
    want, first, out = (torch.full((rows, V), 7.0, dtype=BF, device="cuda") for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_logits_adjust(want, x, row_seq=_i32(seq), allowed=sets, allowed_rows=none, dev_status=st)
    seq[[1, 4]] = -1
    abi.lora_logits_adjust(first, x, row_seq=_i32(seq), allowed=sets, allowed_rows=none, dev_status=st)
    assert abi.lora_read_device_status(st) == 0
    seq[[2, 5]] = -2, LOW
    seq[3] = TOP                                 # without rules there is no last request
    abi.lora_logits_adjust(out, x, row_seq=_i32(seq), allowed=sets, allowed_rows=none, dev_status=st)
    assert abi.lora_read_device_status(st) == abi.LORA_DEV_BAD_SEGMENT
    assert (first[[1, 4]] == 7).all() and (out[[1, 2, 4, 5]] == 7).all()
    keep = [t for t in range(rows) if t not in (1, 2, 4, 5)]
    assert torch.equal(out[keep], want[keep]) and torch.equal(first[keep], want[keep])
