"""The weights' gradients of norm and rotation over all numbers of the grid's CTAs, in a workspace of exactly the size asked for.
Tolerances as those of the small sizes."""
import pytest
import torch

from test_gpu_rotary import BF16, F32, TOL, exact, lib, make, off  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,T", [(128, 1), (128, 8), (128, 9), (128, 16), (128, 17), (128, 2432), (128, 2433), (128, 3000), (128, 4864),
                                 (128, 4865), (16, 64), (16, 129), (64, 5000)])
def test_parts(lib, dtype, d, T):  # noqa: F811
    s = make(dtype, 1, 2, 1, T, d, d, seed=T)
    how = dict(wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"])
    size = lib.mesa_qk_norm_rotary_backward_workspace_size(1, 2, 1, T, d)
    room = torch.full((size + 1024,), 85, dtype=torch.uint8, device="cuda")
    got = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], **how, workspace=room[:size])
    assert bool((room[size:] == 85).all())
    for n, x, y in zip(("q", "k", "wq", "wk"), got, exact(s, False, True, 1.0, 0, grads=True)):
        if n in "qk":
            assert off(x, y) <= 2 * TOL[dtype], n
        else:
            assert float((x.double() - y).norm()) <= 2.0 ** -16 * max(float(s["d" + n[1]].double().norm()), float(y.norm())), n
