"""The convolution's gradients where heads and channels fill the grid by themselves: a thread then adds up whole sequences, a
quarter of all tokens, one after the other.

Sums of dw and dbias: N = B T / 4 terms in one fp32 chain.  An addition is off by at most 2^-24 of the sum so far, which for terms
of independent signs is sqrt(n) of a term's size after n of them; the roundings are independent, so that N of them add up
to sqrt(N^2 / 2) 2^-24 of a term's size, or sqrt(N / 2) 2^-24 of the sum's: 2^-19 at N = 2000, and four chains are added.  SiLU's
derivative from the hardware's exponential and division is 2^-21 of each term: 2^-17."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off
from test_gpu_causal_conv import BF16, F32, TOL, lib  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,W,packed", [(BF16, 4, False), (BF16, 4, True), (F32, 2, True), (BF16, 8, False)])
def test_one_chain_a_thread(lib, dtype, W, packed):  # noqa: F811
    B, H, T, d = 2, 64, 3001, 2048  # (sixteen parts of a head's channels: 1024 CTAs)
    g = torch.Generator(device="cuda").manual_seed(W)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x, dout = (normal(B, H, T, d).to(dtype) for _ in range(2))
    w, bias = W ** -0.5 * normal(H, d, W), 0.3 * normal(H, d)
    starts = torch.rand((B, T), generator=g, device="cuda") < 0.01 if packed else None
    dx, dw, db = lib.mesa_causal_conv_backward(x, w, dout, bias=bias, starts=starts)
    for h in (0, 31, 63):
        t = [y[:, h:h + 1].double().requires_grad_() if y.dim() == 4 else y[h:h + 1].double().requires_grad_() for y in (x, w, bias)]
        out, _ = ref.conv(*t, True, starts)
        (out * dout[:, h:h + 1].double()).sum().backward()
        assert off(dx[:, h:h + 1], t[0].grad) <= TOL[dtype]
        size = float((dout[:, h].double().square().sum() * (1 + x[:, h].double().square().mean())).sqrt())
        for got, want in ((dw[h:h + 1], t[1].grad), (db[h:h + 1], t[2].grad)):
            assert float((got.double() - want).norm()) <= 2.0 ** -17 * max(size, float(want.norm()))
