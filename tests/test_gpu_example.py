"""The example decoder: it learns, and its token-by-token logits are those of the whole sequence."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


# bf16 activations are rounded (2^-9) about ten times per block on either way: a few 1e-2 at most;
# fp32 accumulates 2^-24 over sums of a few hundred terms in a handful of layers: 1e-4 at most (matrix
# products in full fp32).
@pytest.mark.parametrize("dtype,tol", [("bf16", 5e-2), ("f32", 1e-4)])
def test_example_trains_and_decodes(dtype, tol):
    import torch

    from mesa_layer_gb300 import build
    build.build()
    import delta_block as ex
    torch.manual_seed(0)
    model = ex.Decoder(dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, d=128 if dtype == "bf16" else 64)
    losses = ex.train(model, 30)
    assert losses[-1] < losses[0] - 0.2, losses
    x = ex.recall_batch(2, 150, 64, 99)
    with torch.no_grad():
        whole = model(x)
    _, memory = model.prefill(x[:, :131])
    for t in range(131, 150):
        logits = model.step(memory, x[:, t])
        assert float((logits - whole[:, t]).norm() / whole[:, t].norm()) <= tol


def test_example_gradients_against_plain_autograd():
    """One fp32 block's parameter gradients against the same block written with plain operations in
    64 bits (2^-24 over sums of a few hundred terms, through two norms: 1e-4)."""
    import torch
    import torch.nn.functional as F

    import delta_block as ex
    model = ex.Decoder(vocab=16, layers=1, H=2, Hk=1, d=32, dtype=torch.float32)
    x = ex.recall_batch(2, 70, 16, 3)
    F.cross_entropy(model(x)[:, :-1].flatten(0, 1), x[:, 1:].flatten()).backward()
    got = [p.grad.double() for p in model.parameters()]

    ps = [p.detach().double().requires_grad_() for p in model.parameters()]
    embed, head, first = ps[:3]
    b = dict(zip(model.blocks[0], ps[3:]))

    def rms(y):
        return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)

    def heads(t, n):
        return t.view(2, 70, n, -1).transpose(1, 2)

    r = embed[x]
    h = rms(r) * first
    before = torch.cat((torch.zeros_like(h[:, :1]), h[:, :-1]), 1)
    q, k = (F.normalize(heads(t @ b[n], 1), dim=-1, eps=1e-6) for t, n in ((h, "q"), (before, "k")))
    a, beta = heads(h @ b["ab"], 4)[..., 0].chunk(2, 1)
    gamma, beta, v = torch.sigmoid(a + 4.0), torch.sigmoid(beta), heads(h @ b["v"], 2)
    S, outs = torch.zeros(2, 2, 32, 32, dtype=torch.float64, device="cuda"), []
    for t in range(70):
        kt, qt = k[:, :, t].expand(-1, 2, -1), q[:, :, t].expand(-1, 2, -1)
        S = gamma[:, :, t, None, None] * S
        e = v[:, :, t] - (S @ kt[..., None])[..., 0]
        S = S + (beta[:, :, t, None] * e)[..., None] * kt[:, :, None]
        outs.append(32 ** -0.5 * (S @ qt[..., None])[..., 0])
    o = rms(torch.stack(outs, 2)) * b["w_head"] * F.silu(heads(h @ b["gate"], 2))
    r = r + b["res_scale"] * (o.transpose(1, 2).reshape(2, 70, 64) @ b["o"])
    logits = (rms(r) * b["w_pre"]) @ head
    F.cross_entropy(logits[:, :-1].flatten(0, 1), x[:, 1:].flatten()).backward()
    for g, p in zip(got, ps):
        assert float((g - p.grad).norm() / p.grad.norm()) <= 1e-4
