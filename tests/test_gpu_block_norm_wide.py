"""Block norm rows of 2049 to 4096 channels (512 threads a row) beside the widths of test_gpu_block_norm.py,
with its checks and tolerances."""
import pytest

import test_gpu_block_norm as base
from test_gpu_block_norm import ALL, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = [("f32", 3, 2049, ALL), ("f32", 5, 4096, ALL), ("f32", 400, 2500, dict(gate=1, w_post=1)),
        ("f32", 2, 4095, dict(x=1, w_pre=1)), ("bf16", 3, 2056, ALL), ("bf16", 500, 4096, ALL), ("bf16", 7, 4094, ALL),
        ("bf16", 2, 2051, dict(x=1, w_post=1, w_pre=1))]


@pytest.mark.parametrize("case", WIDE, ids=str)
def test_forward(case):
    base.test_forward(case)


@pytest.mark.parametrize("case", WIDE, ids=str)
def test_backward(case):
    base.test_backward(case)
