"""The chunked 64-bit scan against the token recurrence, gradients and all (CPU)."""
import pytest
import torch

import mixer_reference as ref
import scan_reference as chunks


@pytest.mark.parametrize("T", [1, 9, 16, 37])
@pytest.mark.parametrize("packed", [False, True])
def test_chunks_are_the_recurrence(T, packed):
    g = torch.Generator().manual_seed(T)

    def normal(*shape):
        return torch.randn(*shape, dtype=torch.float64, generator=g)

    B, H, Hk, dk, dv = 2, 4, 2, 3, 5
    x = [normal(B, Hk, T, dk), normal(B, Hk, T, dk), normal(B, H, T, dv), normal(B, H, T), -torch.rand(H, generator=g).double() - 0.1,
         normal(H), normal(H)]
    S0 = normal(B, H, dv, dk)
    starts = torch.rand(B, T, generator=g) < 0.2 if packed else None
    weights = normal(B, H, T, dv), normal(B, H, dv, dk)
    grads = []
    for f in (lambda *a: ref.scan(*a, starts, S), lambda *a: chunks.chunked(*a, starts, S, C=8)[:2]):
        leaves = [t.clone().requires_grad_() for t in (*x, S0)]
        S = leaves[-1]
        out = f(*leaves[:-1])
        sum((o * w).sum() for o, w in zip(out, weights)).backward()
        grads.append([*(o.detach() for o in out), *(t.grad for t in leaves)])
    for a, b in zip(*grads):
        assert torch.allclose(a, b, rtol=1e-9, atol=1e-11)


def test_the_log_decays_gradients_are_the_sums_terms():
    """dA is the sum of step times the log-decays' gradients."""
    torch.manual_seed(1)
    B, H, T = 2, 3, 21
    s = dict(q=torch.randn(B, H, T, 4), k=torch.randn(B, H, T, 4), v=torch.randn(B, H, T, 4), dt=torch.randn(B, H, T),
             A=-torch.rand(H) - 0.1, dt_bias=None, skip=None, starts=torch.rand(B, T) < 0.2, S0=torch.randn(B, H, 4, 4),
             dout=torch.randn(B, H, T, 4), dS_final=torch.randn(B, H, 4, 4))
    g = chunks.gradients(s)
    step = torch.nn.functional.softplus(s["dt"].double())
    assert torch.allclose((step * g["log"]).sum((0, 2)), g["A"]) and not g["log"][:, 0][s["starts"]].any()
    assert torch.allclose(chunks.chunks_shares(step * g["log"], 8).sum((0, 2)), g["A"])
