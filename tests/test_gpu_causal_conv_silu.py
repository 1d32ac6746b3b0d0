"""SiLU of fp32 calls to fp32's last bits.

One tap of 1 and no bias: y is x, and out = y sigmoid(y).  The exponential is off by 2^-22.5 (what its argument's rounding leaves
out is put back), one plus it by 2^-24, the reciprocal by 2^-23, the product by 2^-24: together below 2^-21, as long as the
result is above 2^-120 (y >= -83).  Gradients: g (1 + y (1 - g)), whose 1 - g has the rounding of a g close to one, 2^-22 at
most, so that y g 2^-22 comes on top of 2^-21 of the terms' size."""
import pytest
import torch

from test_gpu_causal_conv import lib  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def test_values(lib):  # noqa: F811
    y = torch.linspace(-83, 83, 1 << 20, device="cuda")
    y = torch.cat([y, torch.linspace(-2, 2, 1 << 18, device="cuda")]).view(1, 1, -1, 8).contiguous()
    w = torch.ones(1, 8, 1, device="cuda")
    x = y.double()
    g = torch.sigmoid(x)
    out = lib.mesa_causal_conv(y, w).double()
    assert bool(((out - x * g).abs() <= 2.0 ** -21 * (x * g).abs()).all())
    step = lib.mesa_causal_conv_step(y[0, 0, :, None].contiguous(), w, None).double()
    assert torch.equal(step[:, 0], out[0, 0])
    dx, _, _ = lib.mesa_causal_conv_backward(y, w, torch.ones_like(y))
    bound = 2.0 ** -21 * g * (1 + x.abs() * (1 - g)) + 2.0 ** -22 * g * x.abs()
    assert bool(((dx.double() - g * (1 + x * (1 - g))).abs() <= bound).all())


def test_infinities(lib):  # noqa: F811
    y = torch.tensor([torch.inf, -torch.inf, torch.nan, 3e38, -3e38, 0.0, -0.0, 1e-40], device="cuda").view(1, 1, 1, 8)
    out = lib.mesa_causal_conv(y, torch.ones(1, 8, 1, device="cuda"))[0, 0, 0]
    want = y[0, 0, 0].double()
    want = want * torch.sigmoid(want)
    assert out[0] == torch.inf and out[1:3].isnan().all() and torch.equal(out[3:], want[3:].float())
