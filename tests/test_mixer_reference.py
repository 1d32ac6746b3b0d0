"""The 64-bit forms of the scan, the convolution and the norm and rotation: against differences, and against what has to
hold of them (CPU)."""
import pytest
import torch

import mixer_reference as ref


def _normal(*shape):
    return torch.randn(*shape, dtype=torch.float64)


@pytest.mark.parametrize("packed", [False, True])
def test_scan_gradients_are_differences(packed):
    torch.manual_seed(0)
    B, H, Hk, T, dk, dv = 2, 4, 2, 5, 3, 2
    x = [_normal(B, Hk, T, dk), _normal(B, Hk, T, dk), _normal(B, H, T, dv), _normal(B, H, T), -torch.rand(H).double() - 0.1,
         _normal(H), _normal(H), _normal(B, H, dv, dk)]
    starts = torch.tensor([[0, 0, 1, 0, 0], [1, 0, 0, 0, 1]]).bool() if packed else None
    x = [t.requires_grad_() for t in x]
    f = lambda q, k, v, dt, A, b, s, S0: ref.scan(q, k, v, dt, A, b, s, starts, S0)  # noqa: E731
    assert torch.autograd.gradcheck(f, x)


def test_scan_start_is_a_new_sequence():
    torch.manual_seed(1)
    T, cut = 9, 4
    q, k, v, dt = _normal(1, 1, T, 4), _normal(1, 1, T, 4), _normal(1, 1, T, 3), _normal(1, 1, T)
    A, S0 = -torch.ones(1).double(), _normal(1, 1, 3, 4)
    starts = torch.zeros(1, T).bool()
    starts[0, cut] = True
    out, S = ref.scan(q, k, v, dt, A, starts=starts, S0=S0)
    first, _ = ref.scan(q[:, :, :cut], k[:, :, :cut], v[:, :, :cut], dt[:, :, :cut], A, S0=S0)
    second, S2 = ref.scan(q[:, :, cut:], k[:, :, cut:], v[:, :, cut:], dt[:, :, cut:], A)
    assert torch.equal(out, torch.cat([first, second], 2)) and torch.equal(S, S2)


def test_scan_padding_leaves_the_state():
    torch.manual_seed(2)
    q, k, v, dt = _normal(1, 1, 6, 4), _normal(1, 1, 6, 4), _normal(1, 1, 6, 3), _normal(1, 1, 6)
    A = -torch.ones(1).double()
    dt[0, 0, 4:] = -torch.inf
    assert torch.equal(ref.scan(q, k, v, dt, A)[1], ref.scan(q[:, :, :4], k[:, :, :4], v[:, :, :4], dt[:, :, :4], A)[1])


@pytest.mark.parametrize("W", [1, 3])
def test_conv_gradients_are_differences(W):
    torch.manual_seed(3)
    x = [t.requires_grad_() for t in (_normal(2, 2, 6, 3), _normal(2, 3, W), _normal(2, 3))]
    starts = torch.tensor([[0, 0, 1, 0, 0, 0], [0, 1, 1, 0, 0, 0]]).bool()
    assert torch.autograd.gradcheck(lambda x, w, b: ref.conv(x, w, b, True, starts)[0], x)


def test_conv_goes_on_from_its_state():
    torch.manual_seed(4)
    x, w, b = _normal(1, 2, 11, 3), _normal(2, 3, 4), _normal(2, 3)
    whole, end = ref.conv(x, w, b)
    first, state = ref.conv(x[:, :, :2], w, b)
    second, end2 = ref.conv(x[:, :, 2:], w, b, state0=state)
    assert torch.equal(whole, torch.cat([first, second], 2)) and torch.equal(end, end2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_gradients_are_differences_and_lengths_stay(interleaved):
    torch.manual_seed(5)
    x, w = _normal(2, 2, 3, 8).requires_grad_(), (1 + 0.1 * _normal(8)).requires_grad_()
    f, pos = torch.tensor([1.0, 0.1, 0.01]).double(), torch.tensor([[0, 5, 1000], [7, 8, 9]])
    assert torch.autograd.gradcheck(lambda x, w: ref.rotate(x, w, f, pos, interleaved, 1.1, True, 1e-6), [x, w])
    y = ref.rotate(x, None, f, pos, interleaved, 1.0, False, 0.0)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
    # scalar products go by the distance alone
    a, b = _normal(1, 1, 1, 8), _normal(1, 1, 1, 8)

    def dot(p, q):
        return (ref.rotate(a, None, f, torch.tensor([[p]]), interleaved, 1.0, False, 0.0) *
                ref.rotate(b, None, f, torch.tensor([[q]]), interleaved, 1.0, False, 0.0)).sum()

    assert torch.allclose(dot(3, 10), dot(103, 110))
