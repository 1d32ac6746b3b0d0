"""Row counts past what the C interface's int holds are refused, not wrapped (CPU: a stand-in for the tensor)."""
import types

import pytest
import torch

from mesa_layer_gb300 import binding


class Rows:
    device, dtype, is_cuda = types.SimpleNamespace(index=0), torch.bfloat16, True

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True


def test_block_norm_rows():
    assert binding._norm_check(None, Rows(3, 5, 16), None, None, None, None) == (15, 16)
    assert binding._norm_check(None, Rows(2 ** 31 - 1, 16), None, None, None, None) == (2 ** 31 - 1, 16)
    for shape in ((2 ** 31, 16), (2 ** 32 + 8, 1), (2 ** 16, 2 ** 16, 64)):
        with pytest.raises(binding.MesaError):
            binding._norm_check(None, Rows(*shape), None, None, None, None)
