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


def test_the_longest_sequence(lib):  # noqa: F811
    """2^31 - 256 tokens: a run's first token and its length together pass 32 bits."""
    room(128)
    T, d, W = 0x7fffff00, 8, 2
    x, dout, dx = (torch.zeros(1, 1, T, d, dtype=BF16, device="cuda") for _ in range(3))
    w = torch.tensor([1.0, 2.0], device="cuda").expand(1, d, W).contiguous()
    at = torch.tensor([0, 1, T // 2, T - 60000, T - 1000, T - 2, T - 1], device="cuda")
    x[0, 0, at], dout[0, 0, at] = 3.0, 1.0
    dx.fill_(7.0)
    _, dw, _ = lib.mesa_causal_conv_backward(x, w, dout, silu=False, dx=dx)
    assert torch.equal(dw[0, 0], torch.tensor([21.0, 6.0], device="cuda"))  # (two of them have one right before)
    # dx_t = dout_t + 2 dout_{t+1}
    for a, b in ((0, 1 << 20), (T // 2 - 1000, T // 2 + 1000), (T - (1 << 20), T)):
        piece = dout[0, 0, a:b].float()
        piece[:-1] += 2 * dout[0, 0, a + 1:b].float()
        if b < T:
            piece[-1] += 2 * dout[0, 0, b].float()
        assert torch.equal(dx[0, 0, a:b].float(), piece)
    assert not (dx == 7.0).any()
    out = lib.mesa_causal_conv(x, w, silu=False, out=dx)  # (and the forward: x_t + 2 x_{t-1})
    assert torch.equal(out[0, 0, T - 3:].float(), torch.tensor([0.0, 3.0, 9.0], device="cuda")[:, None].expand(3, d))
    assert float(out[0, 0, 0, 0]) == 3.0 and float(out[0, 0, 1, 0]) == 9.0
