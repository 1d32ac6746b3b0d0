"""The scan's gradients where packed documents differ in loudness: nothing of one reaches another's.

Tolerances on the 2-norm of each document's own values: those of the gradients elsewhere (fp32: 2^-15 over sums of a few
hundred terms; bf16: 4 2^-8, the output's rounding and that of three operands).  Where a document's dout is zero every term
of its steps' gradients is a product with zero: exactly zero."""
import pytest
import torch

from test_gpu_ssm import BF16, F32, GRAD_TOL, exact, lib, make  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu
SIZES = [(F32, 32, 32), (F32, 64, 64), (BF16, 128, 128), (BF16, 128, 64), (BF16, 64, 64), (BF16, 32, 32)]
CUTS = [(128, [64]), (128, [1, 40, 41, 100]), (300, [5, 37, 130, 150, 256])]


def packed(dtype, dk, dv, T, cuts, seed):
    s = make(dtype, 2, 4, 2, T, dk, dv, seed=seed, steps=(1e-3, 1e-1))
    s["starts"] = torch.zeros(2, T, dtype=torch.bool, device="cuda")
    s["starts"][:, cuts] = True
    return s, list(zip([0, *cuts], [*cuts, T]))


def backward(lib, s):  # noqa: F811
    return lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"],
                                         starts=s["starts"], gates_dtype=F32)


@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("T,cuts", CUTS)
@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_silent_documents(lib, dtype, dk, dv, T, cuts, first):  # noqa: F811
    s, documents = packed(dtype, dk, dv, T, cuts, T + first)
    for a, b in documents[first::2]:
        s["dout"][:, :, a:b] = 0
    got = backward(lib, s)
    for a, b in documents[first::2]:
        assert all(not x[:, :, a:b].any() for x in got[:4])


@pytest.mark.parametrize("loud", [1e4, 1e6])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("T,cuts", CUTS)
@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_quiet_documents_beside_loud_ones(lib, dtype, dk, dv, T, cuts, first, loud):  # noqa: F811
    s, documents = packed(dtype, dk, dv, T, cuts, T + first)
    for a, b in documents[first::2]:
        s["dout"][:, :, a:b] *= loud
    want, got = exact(s, grads=True), backward(lib, s)
    for n, x in zip(("q", "k", "v", "dt"), got):
        for a, b in documents:
            y = want[n][:, :, a:b]
            assert float((x[:, :, a:b].double() - y).norm()) <= GRAD_TOL[dtype] * float(y.norm()), (n, a, b)
