"""The convolution's gradients at sizes whose indices pass 32 bits: of the weights' sums, of the tokens.

Inputs are zero but where they are looked at, small whole numbers there, so that every value is exact."""
import pytest
import torch

from test_gpu_causal_conv import BF16, F32, lib  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"{gigabytes} GB of free memory are needed")


@pytest.mark.parametrize("H", [911, 1024, 4096])  # 2^29 and 2^31 sums, and more
def test_sums_of_many_channels(lib, H):  # noqa: F811
    room(8 * H // 1024 + 4)
    d, W = 65536, 8
    x, dout = (torch.zeros(1, H, 1, d, dtype=BF16, device="cuda") for _ in range(2))
    w, bias = torch.zeros(H, d, W, device="cuda"), torch.zeros(H, d, device="cuda")
    dw, dbias = torch.full_like(w, torch.nan), torch.full_like(bias, torch.nan)
    for h in (0, 1, H // 2, H - 2, H - 1):
        x[0, h, 0] = torch.arange(d, device="cuda") % 13 + 1
        dout[0, h, 0] = h % 5 + 1
    lib.mesa_causal_conv_backward(x, w, dout, bias=bias, silu=False, dw=dw, dbias=dbias)
    assert not dw[..., 1:].any()  # (taps before the first token)
    assert torch.equal(dw[..., 0], x[0, :, 0].float() * dout[0, :, 0].float()) and torch.equal(dbias, dout[0, :, 0].float())
