"""The attention block of examples/attention_block.py: prompts and then single
tokens give what one pass over the whole sequences gives.

The two ways differ in the roundings of the projections (another kernel by
the number of rows), which move a cached value across a step's boundary now
and then: 2^-8 of the values in bf16, a step of a fifteenth of a group's
range where a code flips, so that the outputs agree to a few percent."""
import importlib.util
import os

import pytest
import torch

from lora_serving_gb300 import abi, build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    build()
    abi.load()
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("shape", [dict(hidden=512, heads=8, kv=2, dim=64, prompts=(130, 3, 65), steps=7, page=16),
                                   dict(hidden=1024, heads=6, kv=2, dim=128, prompts=(300, 17), steps=5, page=64)])
def test_steps_give_what_one_pass_gives(example, shape):
    assert example.run(**shape) < 0.05
