"""Steps that forget all that went before, several within a few tokens, among small ones: the decays between the small ones stay
exact however large the logarithms' sums have become (2^-150 a reset, so that thirty of them reach 4500, of which an fp32 unit
is 2^-11).

One group of 32 tokens, no state before it and none after: each step's gradient is a sum of pairs in fp32.  A pair is a product
of two sums of at most 128 products of bf16 values (exact products, 2^-24 a sum's step: 2^-17), a decay (the hardware's
exponential, 2^-22, of a difference that is 2^-21 off) and a step (2^-23); 31 x 31 pairs are added (2^-18 of their size at
most).  2^-15 in all, measured on the sum of the pairs' absolute values by their 2-norm; CUDA cores alike.  The outputs are
rounded to bf16 and their weights were: 3 2^-8 as elsewhere."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off
from test_gpu_ssm import BF16, F32, TOL, lib, make  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def resets(dtype, dk, dv, T, at, seed):
    s = make(dtype, 1, 4, 2, T, dk, dv, seed=seed, steps=(1e-2, 1e-1))
    s["dt"][:, :, at] = 1e4  # (A <= -1: e^-10000)
    s["v"][:, :, at] = 0
    s["dout"][:, :, at] = 0
    return s


def decays_gradient(s):
    """ddt of the steps' decays and values in 64 bits, and the same of absolute values, [1, H, T] (T small; no states)."""
    B, H, T = s["dt"].shape
    q, k = (s[n].double().repeat_interleave(2, 1) for n in "qk")
    v, g = s["v"].double(), s["dout"].double()
    raw = s["dt"].double() + s["dt_bias"].double()[:, None]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    log = (step * s["A"].double()[:, None]).cumsum(-1)
    low = torch.ones(T, T, device="cuda").tril().bool()
    E = torch.exp(torch.where(low, log[..., :, None] - log[..., None, :], -torch.inf))
    X = (q @ k.mT) * (g @ v.mT) * E  # reader i, writer j, without the writer's step
    out = []
    for x in (X, X.abs()):
        own = x.sum(-2)
        w = x * step[..., None, :]
        da = torch.stack([w[..., t:, :t].sum((-1, -2)) for t in range(T)], -1)
        A = s["A"].double()[:, None]
        out.append((own + (A if x is X else A.abs()) * da) * torch.sigmoid(raw))
    return out


AT = [[3], [0, 1, 2, 3, 4], list(range(0, 24)), list(range(1, 27, 2)) + [2, 4, 6, 8, 10]]


@pytest.mark.parametrize("at", AT, ids=len)
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 32), (F32, 128, 128), (BF16, 128, 128), (BF16, 128, 64), (BF16, 64, 64)])
def test_steps_between_resets(lib, dtype, dk, dv, at):  # noqa: F811
    T = 32
    s = resets(dtype, dk, dv, T, at, seed=len(at))
    ddt = lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"],
                                        gates_dtype=F32)[3]
    want, size = decays_gradient(s)
    small = torch.ones(T, dtype=torch.bool, device="cuda")
    small[at] = False
    assert float((ddt.double() - want)[..., small].norm()) <= 2.0 ** -15 * float(size[..., small].norm())
    out = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"])
    assert off(out, ref.scan(*(s[n].double() for n in ("q", "k", "v", "dt", "A", "dt_bias", "skip")))[0]) <= TOL[dtype]


def test_the_sum_above_is_the_gradient():  # (CPU would do; the inputs are made on the GPU)
    s = resets(F32, 16, 16, 20, [2, 3, 9], seed=1)
    x = {n: s[n].double().requires_grad_() for n in ("q", "k", "v", "dt", "A", "dt_bias", "skip")}
    out, _ = ref.scan(*x.values())
    (out * s["dout"].double()).sum().backward()
    # (three resets of up to 16 e4 each: the logarithms' sums reach 4.8e5, of which a 64-bit unit is 2^-34; a difference of two
    # is off by as much, and so is its exponential)
    assert off(decays_gradient(s)[0], x["dt"].grad) <= 2.0 ** -33
