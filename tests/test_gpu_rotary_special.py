"""Norm and rotation where channels that do not turn hold what is not finite: it stays in its channel (without the norm, in
which every channel of a row takes part)."""
import pytest
import torch

from test_gpu_rotary import BF16, F32, lib, make  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu
BAD = [torch.inf, -torch.inf, torch.nan]


def same(x, y):
    return torch.equal(x.isnan(), y.isnan()) and torch.equal(x[~x.isnan()], y[~y.isnan()])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R", [(64, 32), (128, 64), (128, 16), (32, 12), (16, 6), (64, 0), (64, 62)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_channels_that_do_not_turn(lib, dtype, d, R, interleaved, bad):  # noqa: F811
    s = make(dtype, 2, 3, 2, 11, d, R, seed=R, norm=False)
    how = dict(inv_freq=s["inv_freq"], offset=3, interleaved=interleaved, norm=False)
    clean = lib.mesa_qk_norm_rotary(s["q"], s["k"], **how)
    grads = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], **how)
    for channel in {R, d - 1, (R + d) // 2}:
        q, dq = s["q"].clone(), s["dq"].clone()
        q[1, 2, 5, channel] = dq[0, 1, 7, channel] = bad
        out = lib.mesa_qk_norm_rotary(q, s["k"], **how)
        want = clean[0].clone()
        want[1, 2, 5, channel] = bad
        assert same(out[0], want) and torch.equal(out[1], clean[1])
        g = lib.mesa_qk_norm_rotary_backward(q, s["k"], dq, s["dk"], **how)
        want = grads[0].clone()
        want[0, 1, 7, channel] = bad
        assert same(g[0], want) and torch.equal(g[1], grads[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_infinity_and_the_norm(lib, dtype, interleaved):  # noqa: F811
    """rsqrt of an infinite mean is 0: the row's finite channels that do not turn are 0, the infinite one is NaN."""
    s = make(dtype, 1, 2, 1, 4, 64, 32, seed=1)
    s["q"][0, 1, 2, 45] = torch.inf
    out = lib.mesa_qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], interleaved=interleaved)[0][0, 1, 2]
    assert out[45].isnan() and not out[:45].any() and not out[46:].any()
