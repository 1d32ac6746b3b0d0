"""Segments of several chunks against the 64-bit scan, and the gates' and parameters' gradients before their rounding.

Tolerances, 2-norms.  Outputs, states and dq, dk, dv as elsewhere (bf16: 3 2^-8, gradients 4 2^-8; fp32 states of bf16 inputs
2^-15).  ddt and the parameters' gradients in fp32: inside a chunk all of it is fp32, products of two sums of at most 128 exact
products (2^-17), decays (2^-21) and steps, added over the chunk: 2^-15.  What passes between chunks goes through states
and adjoints as bf16 operands, each element off by up to 2^-9 of it, 2^-9.2 in the mean, independently of the others: a sum of
products with independent signs is off by that share of its root-sum-square, <R, S> with both rounded by 2^-8.7.  Over n
such sums (chunks of all units) the norms of errors and values are those of n independent normal numbers each: their ratio
passes 2^-8.7 by the root of an F(n, n) number, 1.6 at most for n >= 48 but in one of 1000 cases, so 2^-8.  A parameter's
gradient adds up to 128 tokens of a chunk whose errors are the same rounding's: it is measured on its chunks' shares (2-norm
over batch, heads and chunks of a chunk's sum).  Where a few shares make up most of that norm (a head much more forgetful than
the others, chunks before a document's start), n is that few: (sum x^2)^2 / sum x^4 over n normal numbers is n / 3, so below
16 of it fewer than 48 count; with n = 6 the root is 4.5 at most but in one of 1000 cases: 2^-6.5.  (Two such cases, the norm's
share 4.2e-3 and 4.8e-3: their errors are, head by head, what rounding the states and adjoints of the 64-bit form gives, to
6e-2 and 6e-3 of them.)"""
import pytest
import torch

from scan_reference import chunked, chunks_shares, gradients
from test_gpu_ssm import BF16, F32, GRAD_TOL, STATE_TOL, TOL, lib, make, off  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu
L = 128


def segments(lib, U, T, backward):  # noqa: F811
    """(segments, chunks of one) from the workspaces' sizes: a state of each segment (and an adjoint) of dv columns."""
    size = lib.mesa_ssm_backward_workspace_size if backward else lib.mesa_ssm_workspace_size
    NC, kinds = -(-T // L), 2 if backward else 1
    n = size(1, U, U, T, 128, 128, BF16) - size(1, U, U, T, 128, 64, BF16)
    n -= 2 * U * NC * L * 64 * 2 if backward else 0  # (operand tiles of every chunk)
    assert n % (kinds * U * 64 * 128 * 4) == 0
    n = max(n // (kinds * U * 64 * 128 * 4), 1)
    return n, -(-NC // n)


LONG = [  # B, H, Hk, T, segments of the forward, of the backward
    (1, 16, 16, 20 * L - 3, 7, 7), (2, 24, 6, 9 * L, 3, 1), (3, 10, 5, 32 * L - 5, 5, 5), (1, 2, 1, 300 * L - 77, 75, 75)]
STEPS = [(1e-6, 2e-6), (1e-3, 1e-2), (1e-2, 1e-1), (0.5, 1.0)]


def case(B, H, Hk, T, dk, dv, steps, packed, skip=False):
    s = make(BF16, B, H, Hk, T, dk, dv, seed=T + dv, states=True, steps=steps, skip=skip)
    if packed:  # documents that begin inside segments and chunks, and where one begins
        s["starts"] = torch.zeros(B, T, dtype=torch.bool, device="cuda")
        s["starts"][:, [5 * L + 40, 8 * L, 8 * L + 1]] = True
        s["starts"][-1, 4 * L + 127] = True
    return s


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("B,H,Hk,T,n,m", LONG)
def test_forward(lib, B, H, Hk, T, n, m, dk, dv, steps, packed):  # noqa: F811
    got_n, per = segments(lib, B * H, T, False)
    assert got_n == n and per > 1
    s = case(B, H, Hk, T, dk, dv, steps, packed)
    S = torch.empty_like(s["S0"])
    out = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], starts=s["starts"], S0=s["S0"], S_final=S)
    want, want_S, _ = chunked(*(s[x].double() for x in ("q", "k", "v", "dt", "A", "dt_bias")), starts=s["starts"], S0=s["S0"].double())
    for b, e in ((0, T), (0, T // 2), (T // 2, T)):
        assert off(out[:, :, b:e], want[:, :, b:e]) <= TOL[BF16]
    assert off(S, want_S) <= STATE_TOL[BF16]


def check_gates(s, got, want, tol):
    """ddt and the parameters' gradients, not rounded."""
    raw = s["dt"].double() + (0 if s["dt_bias"] is None else s["dt_bias"].double()[:, None])
    step = torch.nn.functional.softplus(raw)
    assert off(got["dt"], want["dt"]) <= tol
    terms = {"A": step * want["log"], "dt_bias": want["dt"], "skip": (s["dout"].double() * s["v"].double()).sum(-1)}
    for n, x in terms.items():
        if s[n] is not None:
            shares = chunks_shares(x)
            few = float(shares.square().sum() ** 2) < 16 * float(shares.pow(4).sum())
            bound = 2.0 ** -15 if n == "skip" else 2.0 ** -6.5 if tol == 2.0 ** -8 and few else tol
            assert float((got[n].double() - want[n]).norm()) <= bound * float(shares.norm()), n


def backward(lib, s, **kw):  # noqa: F811
    return dict(zip(("q", "k", "v", "dt", "A", "dt_bias", "skip"), lib.mesa_ssm_backward_chunked(
        s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"], starts=s["starts"], S0=s["S0"],
        dS_final=s["dS_final"], gates_dtype=F32, **kw)))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("B,H,Hk,T,n,m", LONG)
def test_backward(lib, B, H, Hk, T, n, m, dk, dv, steps, packed):  # noqa: F811
    got_m, per = segments(lib, B * H, T, True)
    assert got_m == m and (per > 1 or m == 1)
    s = case(B, H, Hk, T, dk, dv, steps, packed)
    dS0 = torch.empty_like(s["S0"])
    got, want = backward(lib, s, dS0=dS0), gradients(s)
    for x in ("q", "k", "v"):
        for b, e in ((0, T), (0, T // 2), (T // 2, T)):
            assert off(got[x][:, :, b:e], want[x][:, :, b:e]) <= GRAD_TOL[BF16], x
    assert off(dS0, want["S0"]) <= STATE_TOL[BF16]
    check_gates(s, got, want, 2.0 ** -8)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 70, 127, 128])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 32, 64), (F32, 128, 128), (BF16, 128, 128), (BF16, 128, 64), (BF16, 64, 64), (BF16, 32, 32)])
def test_gates_gradients_in_one_chunk(lib, dtype, dk, dv, packed, T):  # noqa: F811
    """All of them fp32: not what a product with rounded weights would give (1.6e-3)."""
    s = make(dtype, 3, 6, 3, T, dk, dv, seed=T + 2, packed=packed)
    check_gates(s, backward(lib, s), gradients(s), 2.0 ** -15)
