"""Sequences of few (batch, head) units that the tensor-core path cuts into segments (from 100 chunks of 64
tokens on), against the token recurrence in 64 bits (on the GPU, for its speed).  Tolerances: those of
test_gpu_delta.py, whose derivation does not depend on the length."""
import pytest

from test_gpu_delta import SCALE, STATE_TOL, TOL, _long_inputs, err, upload

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dgamma", "dbeta")
H = 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()


def reference(t, backward=False):
    """out, S_final of the recurrence, or its gradients by name (dS0 among them), in fp64 (numpy)."""
    import torch
    B, heads, T, dv = t["v"].shape
    group = heads // t["q"].shape[1]

    def rows(n):  # [T, units, channels]
        x = t[n].double()
        x = x.repeat_interleave(group, dim=1) if n in ("q", "k") else x
        return x.reshape(B * heads, T, -1).transpose(0, 1).contiguous()

    q, k, v, g, gamma, beta = (rows(n) for n in ("q", "k", "v", "dout", "gamma", "beta"))
    U, dk = B * heads, q.shape[-1]

    def state(n):
        return torch.zeros(U, dv, dk, dtype=torch.float64, device="cuda") if t[n] is None else t[n].double().reshape(U, dv, dk)

    def step(S, i):  # S_{i+1} in place of S_i; e_i
        S *= gamma[i][..., None]
        e = v[i] - (S @ k[i][..., None])[..., 0]
        S.baddbmm_((beta[i] * e)[..., None], k[i][:, None])
        return e

    def back(x):
        return x.transpose(0, 1).reshape(B, heads, T, -1).cpu().numpy()

    S, span, saved, out = state("S0").clone(), 64, [], torch.empty_like(v)
    for i in range(T):
        if i % span == 0:
            saved.append(S.clone())
        step(S, i)
        out[i] = SCALE * (S @ q[i][..., None])[..., 0]
    if not backward:
        return back(out), S.view(B, heads, dv, dk).cpu().numpy()
    A = state("dS_final").clone()
    d = {n: torch.empty_like(x) for n, x in zip(GRADS, (q, k, v, gamma, beta))}
    for first in range((T - 1) // span * span, -1, -span):
        states, es = [saved[first // span]], []
        for i in range(first, min(T, first + span)):
            S = states[-1].clone()
            es.append(step(S, i))
            states.append(S)
        for i in range(first + len(es) - 1, first - 1, -1):
            before, after, e = states[i - first], states[i - first + 1], es[i - first]
            d["dq"][i] = SCALE * (after.mT @ g[i][..., None])[..., 0]
            A.baddbmm_(SCALE * g[i][..., None], q[i][:, None])
            du = (A @ k[i][..., None])[..., 0]
            d["dbeta"][i] = (du * e).sum(-1, keepdim=True)
            d["dv"][i] = beta[i] * du
            d["dk"][i] = (A.mT @ (beta[i] * e)[..., None])[..., 0] - gamma[i] * (before.mT @ d["dv"][i][..., None])[..., 0]
            A.baddbmm_(-d["dv"][i][..., None], k[i][:, None])
            d["dgamma"][i] = (A * before).sum((-1, -2))[:, None]
            A *= gamma[i][..., None]
    r = {n: back(x) for n, x in d.items()}
    for n in ("dq", "dk"):
        r[n] = r[n].reshape(B, heads // group, group, T, dk).sum(2)
    return {**r, "dS0": A.view(B, heads, dv, dk).cpu().numpy()}


def run(t, backward=False):
    """(outputs by name, (status code, flags))."""
    import torch

    from mesa_layer_gb300 import binding
    B, heads, T, dv = t["v"].shape
    size = binding.mesa_delta_backward_workspace_size if backward else binding.mesa_delta_workspace_size
    ws = torch.empty(size(B, heads, t["q"].shape[1], T, 128, 128, torch.bfloat16), dtype=torch.uint8, device="cuda")
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    state = torch.full((B, heads, dv, 128), float("nan"), device="cuda")
    if backward:
        got = binding.mesa_delta_backward_chunked(*args, t["dout"], SCALE, S0=t["S0"], dS_final=t["dS_final"], dS0=state,
                                                  workspace=ws)
        r = dict(zip((*GRADS, "dS0"), (*got, state)))
    else:
        r = {"out": binding.mesa_delta_forward_chunked(*args, SCALE, S0=t["S0"], S_final=state, workspace=ws), "S_final": state}
    return r, binding.mesa_forward_status_code(ws)


def inputs(T, gates, S0, shared=False, seed=81):
    s = _long_inputs(T, gates, S0, seed)
    if shared:
        s["q"], s["k"] = s["q"][:, :1], s["k"][:, :1]
    return upload(s, "bf16")


LONG = [(6400, "open", True, False), (6465, "kept", True, True), (7000, "loud", False, False), (7001, "mixed", True, False),
        (6999, "kept", False, False), (12111, "open", False, True)]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_forward(case):
    T, gates = case[:2]
    t = inputs(*case)
    got, status = run(t)
    assert status == (0, 0)
    o, S = reference(t)
    if gates == "loud":  # (token norms span 2^30: by parts)
        assert max(err(got["out"][:, :, i:i + 64], o[:, :, i:i + 64]) for i in range(0, T, 64)) <= TOL["bf16"]
    assert err(got["out"], o) <= TOL["bf16"]
    assert err(got["S_final"], S) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_gradients(case):
    T, gates, S0, shared = case
    t = inputs(T, "open" if gates == "loud" else gates, S0, shared)
    parts = [slice(0, T)]
    if gates == "loud":  # dL/dout 2^30 louder in the second half, still there long before it
        t["gamma"].copy_(0.985 + 0.015 * t["beta"])
        t["dout"][:, :, T // 2:] *= 2.0 ** 15
        t["dout"][:, :, :T // 2] *= 2.0 ** -15
        parts = [slice(i, i + 64) for i in range(0, T, 64)]
    got, status = run(t, True)
    assert status == (0, 0)
    want = reference(t, True)
    names = GRADS if gates != "loud" else GRADS[:3]
    found = {n: max(err(got[n][:, :, p], want[n][:, :, p]) for p in parts) for n in names}
    assert max(found.values()) <= TOL["bf16"], found
    assert err(got["dS0"], want["dS0"]) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("what", ["v", "beta", "S0", "dout", "dS_final"])
def test_nonfinite_values_last(what):
    """A NaN early (for the gradients: late) in a long sequence is still there at its other end, 0.95 ^ 6500 of
    it, and reported; the other head keeps its bits."""
    from mesa_layer_gb300 import binding
    t = inputs(6501, "open", True)
    backward = what[0] == "d"
    clean, _ = run(t, backward)
    if what == "v":
        t["v"][0, 1, 70, 5] = float("inf")
    elif what == "beta":
        t["beta"][0, 1, 70] = float("nan")
    elif what == "dout":
        t["dout"][0, 1, 6450, 5] = float("nan")
    else:
        t[what][0, 1, 5, 7] = float("nan")
    got, status = run(t, backward)
    assert status == (binding.MESA_ERR_NONFINITE, 2)
    for n in got:
        assert got[n][0, 0].equal(clean[n][0, 0])
    if backward:
        assert not got["dS0"][0, 1, 5].isfinite().any() and not got["dv"][0, 1, 0, 5].isfinite()
    else:
        assert not got["S_final"][0, 1, 5].isfinite().any() and not got["out"][0, 1, -1, 5].isfinite()


def test_final_states_may_replace_the_first():
    from mesa_layer_gb300 import binding
    t = inputs(6700, "kept", True, True)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    want, _ = run(t)
    S = t["S0"].clone()
    assert binding.mesa_delta_forward_chunked(*args, SCALE, S0=S, S_final=S).equal(want["out"]) and S.equal(want["S_final"])
    want, _ = run(t, True)
    A = t["dS_final"].clone()
    got = binding.mesa_delta_backward_chunked(*args, t["dout"], SCALE, S0=t["S0"], dS_final=A, dS0=A)
    assert A.equal(want["dS0"]) and all(x.equal(want[n]) for x, n in zip(got, GRADS))


def test_writes_stay_inside_their_buffers_and_repeat():
    import torch

    from mesa_layer_gb300 import binding
    from test_gpu_canary import Guarded, workspace
    T, td = 6409, torch.bfloat16
    t = inputs(T, "mixed", True)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    wf = workspace(binding.mesa_delta_workspace_size(1, H, H, T, 128, 128, td))
    wb = workspace(binding.mesa_delta_backward_workspace_size(1, H, H, T, 128, 128, td))
    runs = []
    for _ in range(2):
        out, SF, dS0 = Guarded((1, H, T, 128), td), *(Guarded((1, H, 128, 128), torch.float32) for _ in range(2))
        g = [Guarded((1, H, T, 128), td) for _ in range(3)] + [Guarded((1, H, T), td) for _ in range(2)]
        binding.mesa_delta_forward_chunked(*args, out=out.t, S0=t["S0"], S_final=SF.t, workspace=wf.t)
        binding.mesa_delta_backward_chunked(*args, t["dout"], 1.0, t["S0"], t["dS_final"], *(x.t for x in g), dS0=dS0.t,
                                            workspace=wb.t)
        assert all(x.intact() for x in (out, SF, dS0, wf, wb, *g))
        runs.append([x.t for x in (out, SF, dS0, *g)])
    assert all(x.equal(y) for x, y in zip(*runs))


@pytest.mark.parametrize("backward", [False, True])
def test_wait_give_up_reports_timeout(backward):
    from mesa_layer_gb300 import binding
    t = inputs(6500, "kept", True)
    want, status = run(t, backward)
    assert status == (binding.MESA_OK, 0)
    binding.mesa_debug_set_wait_limit(0)
    try:
        _, (code, bits) = run(t, backward)
    finally:
        binding.mesa_debug_set_wait_limit(-1)
    assert code == binding.MESA_ERR_TIMEOUT and bits & 1 and not bits & 4
    got, status = run(t, backward)
    assert status == (binding.MESA_OK, 0)
    assert all(got[n].equal(want[n]) for n in want)
