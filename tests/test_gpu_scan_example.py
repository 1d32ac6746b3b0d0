"""The example decoder of scan blocks: convolution, norm and rotation, scan and block norm together."""
import os
import sys

import pytest
import torch

import mixer_reference as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    from mesa_layer_gb300 import build
    build.build()
    import scan_block
    return scan_block


# bf16 activations are rounded (2^-8 at most) about ten times per block on either way: 5e-2 at most;
# fp32: 2^-24 over sums of a few hundred terms in a handful of layers: 1e-4 at most.
@pytest.mark.parametrize("dtype,tol", [("bf16", 5e-2), ("f32", 1e-4)])
def test_steps_go_on_from_a_prompt(ex, dtype, tol):
    model = ex.Decoder(dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, d=128 if dtype == "bf16" else 64)
    x = ex.recall_batch(2, 150, 64, 99)
    with torch.no_grad():
        whole = model(x)
    first, memory = model.prefill(x[:, :131])
    assert float((first - whole[:, :131]).norm() / whole[:, :131].norm()) <= tol
    for t in range(131, 150):
        logits = model.step(memory, x[:, t])
        assert float((logits - whole[:, t]).norm() / whole[:, t].norm()) <= tol


def test_packed_documents_are_those_documents(ex):
    model = ex.Decoder(dtype=torch.float32, d=32)
    x = ex.recall_batch(1, 200, 64, 5)
    starts = torch.zeros_like(x, dtype=torch.bool)
    cuts = [0, 37, 38, 130, 200]
    starts[0, cuts[:-1]] = True
    with torch.no_grad():
        whole = model(x, starts)
        apart = torch.cat([model(x[:, a:b].contiguous()) for a, b in zip(cuts, cuts[1:])], 1)
    assert float((whole - apart).norm() / apart.norm()) <= 1e-4


def test_it_trains(ex):
    """Every parameter gets a finite gradient in both types, and a step of Adam changes it."""
    for dtype, d in ((torch.bfloat16, 128), (torch.float32, 64)):
        model = ex.Decoder(dtype=dtype, d=d)
        before = [p.detach().clone() for p in model.parameters()]
        losses = ex.train(model, 2)
        assert all(l == l and l < 1e3 for l in losses)
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in model.parameters())
        assert all(not torch.equal(p.detach(), q) for p, q in zip(model.parameters(), before))


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_against_plain_autograd(ex, packed):
    """One fp32 block's parameter gradients against the same block written with plain operations in 64 bits (2^-24 over sums
    of a few hundred terms, through two norms: 1e-4)."""
    import torch.nn.functional as F
    H, Hk, d, T = 2, 1, 32, 70
    model = ex.Decoder(vocab=16, layers=1, H=H, Hk=Hk, d=d, dtype=torch.float32)
    x = ex.recall_batch(2, T, 16, 3)
    starts = None
    if packed:
        starts = torch.zeros_like(x, dtype=torch.bool)
        starts[0, 31] = starts[1, 0] = starts[1, 64] = True
    F.cross_entropy(model(x, starts)[:, :-1].flatten(0, 1), x[:, 1:].flatten()).backward()
    got = [p.grad.double() for p in model.parameters()]

    ps = [p.detach().double().requires_grad_() for p in model.parameters()]
    embed, head, first = ps[:3]
    b = dict(zip(model.blocks[0], ps[3:]))

    def rms(y):
        return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)

    def heads(t, n):
        return t.view(2, T, n, -1).transpose(1, 2)

    at = torch.arange(T, device="cuda").expand(2, T)
    pos = at if starts is None else at - torch.where(starts, at, 0).cummax(-1).values
    r = embed[x]
    h = rms(r) * first
    vqk, _ = ref.conv(heads(h @ b["vqk"], H + 2 * Hk), b["taps"], b["bias"], True, starts)
    v, q, k = vqk.split((H, Hk, Hk), 1)
    q, k = (ref.rotate(t, b["w" + n], model.inv_freq, pos, False, 1.0, True, 1e-6) for t, n in ((q, "q"), (k, "k")))
    o, _ = ref.scan(q, k, v, heads(h @ b["dt"], H)[..., 0], -torch.exp(b["log_A"]), b["dt_bias"], b["skip"], starts)
    gate = heads(h @ b["gate"], H)
    o = rms(o) * b["w_head"] * gate * torch.sigmoid(gate)
    r = r + b["res_scale"] * (o.transpose(1, 2).reshape(r.shape) @ b["o"])
    logits = (rms(r) * b["w_pre"]) @ head
    F.cross_entropy(logits[:, :-1].flatten(0, 1), x[:, 1:].flatten()).backward()
    for name, g, p in zip(("embed", "head", "first", *model.blocks[0]), got, ps):
        assert float((g - p.grad).norm()) <= 1e-4 * float(p.grad.norm()), name
