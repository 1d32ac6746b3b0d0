"""Queries and keys that no value head reads: their gradients are sums of nothing."""
import pytest
import torch

from test_gpu_ssm import BF16, F32, lib  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 64), (BF16, 128)])
def test_gradients_of_nothing_are_zero(lib, dtype, d):  # noqa: F811
    B, Hk, T = 2, 3, 50
    q, k = (torch.randn(B, Hk, T, d, device="cuda").to(dtype) for _ in range(2))
    v, dt, A = torch.empty(B, 0, T, d, dtype=dtype, device="cuda"), torch.empty(B, 0, T, device="cuda"), torch.empty(0, device="cuda")
    dq, dk = torch.full_like(q, torch.nan), torch.full_like(k, torch.nan)
    out = lib.mesa_ssm_forward_chunked(q, k, v, dt, A)
    r = lib.mesa_ssm_backward_chunked(q, k, v, dt, A, v, dt_bias=A, skip=A, dq=dq, dk=dk)
    assert out.shape == v.shape and not dq.any() and not dk.any() and all(x.numel() == 0 for x in r[2:])
