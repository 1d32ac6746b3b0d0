"""The convolution's gradients where rows of threads take several runs of tokens, long and short ones, or whole sequences;
documents that start at the borders of runs and of groups of tokens.  Tolerances as those of the small sizes: a sum over at
most 256 tokens a row, each rounded to 2^-24 of the terms, and the output's own rounding."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off
from test_gpu_causal_conv import BF16, F32, TOL, lib, make  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def check(lib, s):  # noqa: F811
    x, w, b = (s[n].double().requires_grad_() for n in ("x", "w", "bias"))
    out, _ = ref.conv(x, w, b, True, s["starts"])
    (out * s["dout"].double()).sum().backward()
    got = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], bias=s["bias"], starts=s["starts"])
    assert off(got[0], x.grad) <= TOL[s["x"].dtype]
    size = float((s["dout"].double().square().sum() * (1 + s["x"].double().square().mean())).sqrt())
    for g, want in zip(got[1:], (w.grad, b.grad)):
        assert float((g.double() - want).norm()) <= 2.0 ** -16 * max(size, float(want.norm()))
    again = lib.mesa_causal_conv_backward(s["x"], s["w"], s["dout"], bias=s["bias"], starts=s["starts"])
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,H,T,d,W", [(10, 64, 20, 1024, 4), (2, 64, 150, 512, 3), (1, 8, 1000, 128, 4), (3, 40, 97, 256, 8),
                                       (40, 50, 17, 96, 2), (1, 1, 9000, 8, 5), (4, 30, 50, 136, 7)])
def test_runs(lib, dtype, packed, B, H, T, d, W):  # noqa: F811
    check(lib, make(dtype, B, H, T, d, W, seed=T, packed=packed))


@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("every", [1, 2, 4, 5, 16, 31])
def test_documents_of_one_length(lib, W, every):  # noqa: F811
    s = make(BF16, 2, 3, 130, 64, W, seed=every, packed=True)
    s["starts"].zero_()
    s["starts"][0, ::every] = True
    s["starts"][1, every - 1::every] = True
    check(lib, s)
