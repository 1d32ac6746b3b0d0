"""Which sequences are cut into segments (CPU: their states and matrices show in the workspace's size).  Where
a pass over the segments' starts, one over their matrices and the joins cost more than they save, none is."""
import pytest
import torch

from mesa_layer_gb300 import binding


def segmented(U, T, d, dtype):
    """The workspace of U units against their share of as many units as fill the GPU."""
    size = binding.mesa_delta_workspace_size
    return size(1, U, U, T, d, d, dtype) > 512 + U * (size(1, 1216, 1216, T, d, d, dtype) / 1216)


@pytest.mark.parametrize("U,T,want", [
    # us of one chain, of five or more segments: 16 units of 2048 tokens 98, 160; of 4096 183, 196 (nine: 280);
    # one unit of 8192 312, 240 (six; decays fast: 123)
    (1, 1000, False), (16, 2048, False), (1, 4096, False), (16, 4096, False), (8, 6000, False),
    (1, 6400, True), (1, 8192, True), (16, 8192, True), (16, 65536, True), (30, 65536, True), (31, 65536, False)])
def test_tensor_core_sequences(U, T, want):
    assert segmented(U, T, 128, torch.bfloat16) == want


@pytest.mark.parametrize("U,T,d,want", [
    # fp32, us of one scan, of segments: 32 units of 1024 tokens, d 128, 219, 307; 8 units 219, 109; 32 units, d 64, 170, 86
    (32, 1024, 128, False), (32, 8192, 128, False), (128, 2048, 128, False), (8, 1024, 128, True), (1, 256, 128, True),
    (32, 1024, 64, True), (128, 2048, 64, False), (128, 1024, 32, True), (8, 64, 64, False)])
def test_sequences_on_the_cuda_cores(U, T, d, want):
    assert segmented(U, T, d, torch.float32) == want
