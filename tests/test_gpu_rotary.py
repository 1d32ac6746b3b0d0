"""Norms of queries and keys with the position rotation on the GPU against their 64-bit form.

Tolerances on the 2-norm.  fp32: sums of up to 128 products (2^-24 each), the angles' error (2^-24 of a turn, 2^-21 rad) and
the sines': 2^-18.  bf16: the output's rounding, 2^-8.  Weights' gradients: fp32 sums over the rows, 2^-16 of the terms."""
import pytest
import torch

import mixer_reference as ref
from mixer_reference import off

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 2.0 ** -18, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def make(dtype, B, H, Hk, T, d, R, seed=0, positions=None, norm=True, weights=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    s = dict(q=normal(B, H, T, d).to(dtype), k=normal(B, Hk, T, d).to(dtype) if Hk else None,
             wq=1 + 0.2 * normal(d) if norm and weights else None, wk=1 + 0.2 * normal(d) if norm and weights and Hk else None,
             inv_freq=torch.tensor([10000.0 ** (-2 * j / R) for j in range(R // 2)]) if R else None,
             positions=torch.randint(*positions, (B, T), generator=g).to(torch.int32) if positions else None,
             dq=normal(B, H, T, d).to(dtype), dk=normal(B, Hk, T, d).to(dtype) if Hk else None)
    return {n: None if t is None else t.cuda() for n, t in s.items()}


def exact(s, interleaved, norm, rot_scale, offset, eps=1e-6, grads=False):
    pos = s["positions"]
    B, _, T, _ = s["q"].shape
    if pos is None:
        pos = (offset + torch.arange(T, device="cuda"))[None].expand(B, T)
    x = {n: None if s[n] is None else s[n].double().requires_grad_(grads) for n in ("q", "k", "wq", "wk")}
    out = [None if x[n] is None else ref.rotate(x[n], x["w" + n], s["inv_freq"], pos, interleaved, rot_scale, norm, eps) for n in "qk"]
    if not grads:
        return out
    sum((o * s["d" + n].double()).sum() for o, n in zip(out, "qk") if o is not None).backward()
    return [None if t is None else t.grad for t in x.values()]


CASES = [  # B, H, Hk, T, d, R, interleaved, norm, weights, positions, offset, rot_scale
    (1, 1, 1, 1, 16, 16, False, True, True, None, 0, 1.0), (2, 3, 1, 7, 64, 64, False, True, True, None, 5, 1.0),
    (2, 4, 2, 33, 128, 128, True, True, True, (0, 1 << 20), 0, 1.3), (1, 5, 5, 50, 128, 32, False, True, True, (0, 4096), 0, 1.0),
    (1, 2, 0, 19, 32, 8, False, True, True, None, 0, 1.0), (3, 2, 1, 21, 64, 20, False, True, False, None, 7, 0.9),
    (2, 2, 2, 17, 128, 64, True, False, False, (-50, 50), 0, 1.0), (1, 3, 2, 40, 64, 0, False, True, True, None, 0, 1.0),
    (1, 2, 2, 9, 32, 6, True, True, True, (1 << 23, 1 << 24), 0, 1.0), (70, 16, 4, 1, 128, 128, False, True, True, (0, 1 << 20), 0, 1.0),
    (1, 9, 3, 300, 16, 12, False, False, False, None, 1 << 20, 1.0), (1, 2, 1, 6, 64, 64, False, True, True, (2 ** 31 - 9, 2 ** 31 - 1), 0, 1.0),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(lib, dtype, c):
    B, H, Hk, T, d, R, inter, norm, weights, positions, offset, scale = c
    s = make(dtype, B, H, Hk, T, d, R, seed=T, positions=positions, norm=norm, weights=weights)
    how = dict(wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"], positions=s["positions"], offset=offset, interleaved=inter,
               rot_scale=scale, norm=norm)
    got, want = lib.mesa_qk_norm_rotary(s["q"], s["k"], **how), exact(s, inter, norm, scale, offset)
    far = positions is not None and positions[1] > 1 << 24  # angles of pos f with 2^-48 of f: up to 2^-17 rad there
    for x, y in zip(got, want):
        assert (x is None) == (y is None)
        if x is not None:
            assert off(x, y) <= TOL[dtype] + (2.0 ** -17 if far else 0)
    q, k = s["q"].clone(), None if s["k"] is None else s["k"].clone()
    lib.mesa_qk_norm_rotary(q, k, **how, q_out=q, k_out=k)  # in place
    assert torch.equal(q, got[0]) and (k is None or torch.equal(k, got[1]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", CASES[:-1], ids=str)
def test_backward(lib, dtype, c):
    B, H, Hk, T, d, R, inter, norm, weights, positions, offset, scale = c
    s = make(dtype, B, H, Hk, T, d, R, seed=T + 1, positions=positions, norm=norm, weights=weights)
    how = dict(wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"], positions=s["positions"], offset=offset, interleaved=inter,
               rot_scale=scale, norm=norm)
    got = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], **how)
    want = exact(s, inter, norm, scale, offset, grads=True)
    for n, x, y in zip(("q", "k", "wq", "wk"), got, want):
        assert (x is None) == (y is None), n
        if x is None:
            continue
        if n in "qk":
            assert off(x, y) <= 2 * TOL[dtype], n
        else:
            assert float((x.double() - y).norm()) <= 2.0 ** -16 * max(float(s["d" + n[1]].double().norm()), float(y.norm())), n
    dq, dk = s["dq"].clone(), None if s["dk"] is None else s["dk"].clone()
    again = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], dq, dk, **how, dq=dq, dk=dk)  # in place
    assert all((x is None and y is None) or torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_zero_rows_nothing_beyond_and_empty(lib, dtype):
    s = make(dtype, 1, 2, 1, 5, 64, 64)
    s["q"][0, 1] = 0
    n = s["q"].numel()
    room = torch.full((n + 512,), 3.0, dtype=dtype, device="cuda")
    q, _ = lib.mesa_qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], q_out=room[:n].view(s["q"].shape))
    assert not q[0, 1].any() and bool((room[n:] == 3).all())
    e = s["q"][:, :, :0].contiguous()
    assert lib.mesa_qk_norm_rotary(e, inv_freq=s["inv_freq"])[0].shape == e.shape
    r = lib.mesa_qk_norm_rotary_backward(e, None, e, wq=s["wq"], inv_freq=s["inv_freq"])
    assert not r[2].any() and r[1] is None and r[3] is None


def test_captured(lib):
    s, t = make(BF16, 2, 4, 2, 30, 128, 64, seed=1), make(BF16, 2, 4, 2, 30, 128, 64, seed=2)
    how = lambda x: dict(wq=x["wq"], wk=x["wk"], inv_freq=x["inv_freq"])  # noqa: E731
    want = lib.mesa_qk_norm_rotary(t["q"], t["k"], **how(t))
    wg = lib.mesa_qk_norm_rotary_backward(t["q"], t["k"], t["dq"], t["dk"], **how(t))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.mesa_qk_norm_rotary(s["q"], s["k"], **how(s))
        g = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], **how(s))
    for n in ("q", "k", "wq", "wk", "dq", "dk"):
        s[n].copy_(t[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(out + g, want + wg))
