"""The gated delta rule on the GPU against the 64-bit restatement.

Tolerances, per (batch, head) unit on the 2-norm of each output: fp32 -- a token's value is a sum
of products each rounded to 2^-24, over at most a few hundred decayed terms: 2^-24 sqrt(300) ~
1e-6; ten times that.  bf16 -- outputs rounded to 2^-9 relative at most (rms 1.7e-3 of the
value), operands of the tensor-core products to 2^-12: 5e-3.  A gradient of a gate may cancel to
a small value next to its terms, so gate gradients are measured on the unit's norm as well."""
import numpy as np
import pytest

import delta_reference as ref

pytestmark = pytest.mark.gpu
TOL = {"f32": 1e-5, "bf16": 5e-3}
STATE_TOL = {"f32": 1e-5, "bf16": 2e-3}  # fp32 states from operands rounded to 2^-12
SCALE = 0.25


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()


def upload(s, dtype):
    import torch
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    return {n: None if x is None else torch.from_numpy(np.array(x, dtype=np.float32)).cuda().to(
        td if n in ("q", "k", "v", "dout") else torch.float32) for n, x in s.items()}


def err(got, want):
    """Largest over the leading [B, heads] units of the relative 2-norm (absolute on the whole
    tensor's scale where a unit is zero)."""
    got = got.double().cpu().numpy().reshape(*want.shape[:2], -1)
    want = want.reshape(*want.shape[:2], -1)
    assert np.isfinite(got).all()
    floor = 1e-3 * np.sqrt((want ** 2).sum(-1).mean()) + 1e-30
    return (np.linalg.norm(got - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), floor)).max()


FWD = [  # dtype, B, H, Hk, T, dk, dv, gates, states
    ("f32", 1, 1, 1, 1, 16, 16, "open", False),
    ("f32", 2, 3, 3, 33, 16, 32, "packed", True),
    ("f32", 1, 4, 2, 70, 32, 16, "wide", False),
    ("f32", 2, 4, 1, 257, 64, 64, "open", True),
    ("f32", 1, 2, 2, 100, 128, 64, "one", True),
    ("f32", 1, 2, 1, 65, 128, 128, "shut", True),
    ("bf16", 2, 2, 1, 47, 64, 64, "packed", True),
    ("bf16", 1, 2, 2, 31, 32, 128, "wide", False),
    ("bf16", 1, 2, 2, 90, 128, 64, "open", True),
    ("bf16", 1, 1, 1, 1, 128, 128, "open", True),
    ("bf16", 1, 2, 2, 2, 128, 128, "open", False),
    ("bf16", 2, 4, 2, 63, 128, 128, "packed", True),
    ("bf16", 1, 2, 2, 64, 128, 128, "wide", True),
    ("bf16", 1, 3, 1, 65, 128, 128, "open", False),
    ("bf16", 2, 2, 2, 333, 128, 128, "packed", True),
    ("bf16", 1, 2, 2, 200, 128, 128, "one", False),
    ("bf16", 1, 2, 2, 150, 128, 128, "shut", True),
    ("bf16", 1, 1, 1, 2500, 128, 128, "open", True),
    # few units on the CUDA cores: segments of tokens side by side
    ("f32", 1, 2, 1, 256, 16, 32, "open", True),
    ("f32", 1, 3, 3, 777, 32, 32, "packed", True),
    ("f32", 2, 2, 2, 1025, 64, 64, "one", True),
    ("f32", 1, 1, 1, 2048, 128, 128, "open", False),
    ("f32", 1, 1, 1, 500, 64, 16, "wide", True),
    ("bf16", 1, 2, 1, 999, 64, 64, "open", True),
    ("bf16", 1, 1, 1, 400, 128, 32, "shut", True),
]


@pytest.mark.parametrize("case", FWD, ids=str)
def test_forward(case):
    import torch

    from mesa_layer_gb300 import binding
    dtype, B, H, Hk, T, dk, dv, gates, states = case
    s = ref.rule_inputs(11, dtype, B, H, Hk, T, dk, dv, gates, states)
    t = upload(s, dtype)
    SF = torch.full((B, H, dv, dk), float("nan"), device="cuda") if states else None
    ws = torch.empty(binding.mesa_delta_workspace_size(B, H, Hk, T, dk, dv, t["q"].dtype), dtype=torch.uint8,
                     device="cuda")
    out = binding.mesa_delta_forward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], SCALE, S0=t["S0"],
                                             S_final=SF, workspace=ws)
    assert binding.mesa_forward_status(ws) == 0
    o, S = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["S0"])
    assert err(out, o) <= TOL[dtype]
    if states:
        assert err(SF, S) <= STATE_TOL[dtype]


BWD = [
    ("f32", 1, 1, 1, 1, 16, 16, "open", True),
    ("f32", 2, 2, 1, 37, 16, 64, "packed", True),
    ("f32", 1, 4, 2, 65, 32, 32, "wide", False),
    ("f32", 1, 2, 2, 100, 64, 16, "open", True),
    ("f32", 1, 2, 1, 96, 128, 128, "packed", True),
    ("f32", 1, 1, 1, 40, 64, 64, "shut", True),
    ("bf16", 1, 2, 1, 50, 64, 64, "packed", True),
    ("bf16", 1, 2, 2, 1, 128, 128, "open", True),
    ("bf16", 1, 2, 2, 64, 128, 128, "open", False),
    ("bf16", 2, 4, 2, 130, 128, 128, "packed", True),
    ("bf16", 1, 2, 2, 300, 128, 128, "wide", True),
    ("bf16", 1, 2, 2, 190, 128, 128, "one", False),
    ("bf16", 1, 2, 1, 99, 128, 128, "shut", True),
    ("f32", 1, 2, 1, 256, 16, 32, "open", True),
    ("f32", 1, 3, 1, 777, 32, 32, "packed", True),
    ("f32", 1, 1, 1, 1025, 64, 64, "one", True),
    ("f32", 1, 1, 1, 700, 128, 32, "wide", False),
    ("bf16", 1, 2, 1, 600, 64, 64, "open", True),
]


@pytest.mark.parametrize("case", BWD, ids=str)
def test_backward(case):
    import torch

    from mesa_layer_gb300 import binding
    dtype, B, H, Hk, T, dk, dv, gates, states = case
    s = ref.rule_inputs(12, dtype, B, H, Hk, T, dk, dv, gates, states)
    t = upload(s, dtype)
    dS0 = torch.full((B, H, dv, dk), float("nan"), device="cuda") if states else None
    ws = torch.empty(binding.mesa_delta_backward_workspace_size(B, H, Hk, T, dk, dv, t["q"].dtype),
                     dtype=torch.uint8, device="cuda")
    got = dict(zip(("dq", "dk", "dv", "dgamma", "dbeta"), binding.mesa_delta_backward_chunked(
        t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE, S0=t["S0"], dS_final=t["dS_final"], dS0=dS0,
        workspace=ws)))
    assert binding.mesa_forward_status(ws) == 0
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    found = {n: err(x, want[n]) for n, x in got.items()}
    if states:
        assert err(dS0, want["dS0"]) <= STATE_TOL[dtype]
    assert max(found.values()) <= TOL[dtype], found


def test_gradient_against_differences_of_the_forward():
    """A directional derivative of the GPU forward (fp32; central differences of a loss summed in
    fp64: truncation ~ step^2 = 1e-4 relative, rounding 1e-6 / step = 1e-4) against <grad, d>."""
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(13, "f32", 1, 2, 1, 75, 32, 32, "open")
    t = upload(s, "f32")
    g = dict(zip(("q", "k", "v", "gamma", "beta"), binding.mesa_delta_backward_chunked(
        t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE)))
    gen = torch.Generator(device="cuda").manual_seed(5)
    for name in g:
        d = torch.randn(t[name].shape, generator=gen, device="cuda")
        d = d / d.norm() * t[name].norm()
        step = 1e-2

        def loss(x):
            y = {**t, name: (t[name] + x * d).contiguous()}
            o = binding.mesa_delta_forward_chunked(y["q"], y["k"], y["v"], y["gamma"], y["beta"], SCALE)
            return (o.double() * t["dout"].double()).sum().item()

        num = (loss(step) - loss(-step)) / (2 * step)
        ana = (g[name].double() * d.double()).sum().item()
        size = (g[name].double().norm() * d.double().norm()).item()
        assert abs(num - ana) <= 2e-3 * size, (name, num, ana)


@pytest.mark.parametrize("case", [
    ("f32", 1, 1, 1, 16, 16), ("f32", 3, 4, 2, 32, 64), ("f32", 5, 3, 3, 64, 128), ("f32", 2, 2, 1, 128, 16),
    ("bf16", 1, 16, 16, 128, 128), ("bf16", 7, 6, 2, 128, 128), ("bf16", 2, 3, 1, 64, 64), ("bf16", 4, 2, 2, 16, 32)],
    ids=str)
def test_step_matches_the_recurrence(case):
    from mesa_layer_gb300 import binding
    dtype, N, H, Hk, dk, dv = case
    s = ref.rule_inputs(14, dtype, N, H, Hk, 6, dk, dv, "packed", True)
    t = upload(s, dtype)
    S = t["S0"].clone()
    o, SF = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["S0"])
    for i in range(6):
        out = binding.mesa_delta_step(S, *(t[n][:, :, i].contiguous() for n in ("q", "k", "v", "gamma", "beta")),
                                      scale=SCALE)
        assert err(out, o[:, :, i]) <= TOL[dtype]
    assert err(S, SF) <= TOL["f32"]


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_prefix_then_steps_equal_the_whole(dtype, d):
    """Prefill of a prefix, its state handed to the decode steps and to a second prefill."""
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(15, dtype, 2, 2, 2, 140, d, d, "open")
    t = upload(s, dtype)
    whole, SF = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], 1.0)

    def part(a, b):
        return [t[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "gamma", "beta")]

    S = torch.empty(2, 2, d, d, device="cuda")
    o1 = binding.mesa_delta_forward_chunked(*part(0, 77), S_final=S)
    o2 = binding.mesa_delta_forward_chunked(*part(77, 136), S0=S, S_final=S)  # in place
    outs = [o1, o2] + [binding.mesa_delta_step(S, *(x[:, :, 0].contiguous() for x in part(i, i + 1)))[:, :, None]
                       for i in range(136, 140)]
    assert err(torch.cat(outs, 2), whole) <= TOL[dtype]
    assert err(S, SF) <= STATE_TOL[dtype]


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_same_bits_twice_and_on_another_stream(dtype, d):
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(16, dtype, 2, 4, 2, 150, d, d, "packed")
    t = upload(s, dtype)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]

    def both(stream=None):
        return [binding.mesa_delta_forward_chunked(*args, stream=stream),
                *binding.mesa_delta_backward_chunked(*args, t["dout"], stream=stream)]

    a, b = both(), both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = both(side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_writes_stay_inside_their_buffers(dtype, d):
    import torch

    from mesa_layer_gb300 import binding
    from test_gpu_canary import Guarded, workspace
    B, H, Hk, T = 1, 4, 2, 129
    s = ref.rule_inputs(17, dtype, B, H, Hk, T, d, d, "open", True)
    t = upload(s, dtype)
    td = t["q"].dtype
    g = {n: Guarded(t[n].shape, td) for n in ("q", "k", "v")}
    gates = [Guarded((B, H, T), td) for _ in range(2)]
    out, SF, dS0 = Guarded((B, H, T, d), td), Guarded((B, H, d, d), torch.float32), Guarded((B, H, d, d), torch.float32)
    wf = workspace(binding.mesa_delta_workspace_size(B, H, Hk, T, d, d, td))
    wb = workspace(binding.mesa_delta_backward_workspace_size(B, H, Hk, T, d, d, td))
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    binding.mesa_delta_forward_chunked(*args, out=out.t, S0=t["S0"], S_final=SF.t, workspace=wf.t)
    binding.mesa_delta_backward_chunked(*args, t["dout"], S0=t["S0"], dS_final=t["dS_final"], dq=g["q"].t, dk=g["k"].t,
                                        dv=g["v"].t, dgamma=gates[0].t, dbeta=gates[1].t, dS0=dS0.t, workspace=wb.t)
    st, so = Guarded((B, H, d, d), torch.float32, t["S0"]), Guarded((B, H, d), td)
    binding.mesa_delta_step(st.t, *(x[:, :, 0].contiguous() for x in args), out=so.t)
    for b in [*g.values(), *gates, out, SF, dS0, wf, wb, st, so]:
        assert b.intact()


def test_empty_sequences_pass_the_state_through():
    import torch

    from mesa_layer_gb300 import binding
    q, g = torch.zeros(1, 2, 0, 32, device="cuda"), torch.zeros(1, 2, 0, device="cuda")
    S0, S = torch.randn(1, 2, 32, 32, device="cuda"), torch.empty(1, 2, 32, 32, device="cuda")
    assert binding.mesa_delta_forward_chunked(q, q, q, g, g, S0=S0, S_final=S).numel() == 0
    assert torch.equal(S, S0)
    binding.mesa_delta_forward_chunked(q, q, q, g, g, S_final=S)
    assert not S.any()
    binding.mesa_delta_backward_chunked(q, q, q, g, g, q, dS_final=S0, dS0=S)
    assert torch.equal(S, S0)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_nonfinite_values_stay_in_their_unit_and_are_reported(dtype, d):
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(18, dtype, 1, 3, 3, 200, d, d, "open")
    t = upload(s, dtype)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    clean = binding.mesa_delta_forward_chunked(*args)
    t["v"][0, 1, 150, 3] = float("nan")
    ws = torch.empty(binding.mesa_delta_workspace_size(1, 3, 3, 200, d, d, t["q"].dtype), dtype=torch.uint8,
                     device="cuda")
    out = binding.mesa_delta_forward_chunked(*args, workspace=ws)
    assert binding.mesa_forward_status_code(ws) == (binding.MESA_ERR_NONFINITE, 2)
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[0, 2], clean[0, 2])
    assert torch.equal(out[0, 1, :128], clean[0, 1, :128])
    assert out[0, 1, 150, 3].isnan()


def test_bad_shapes_are_refused():
    import torch

    from mesa_layer_gb300 import binding
    q, v = torch.zeros(1, 2, 4, 16, device="cuda"), torch.zeros(1, 3, 4, 16, device="cuda")
    g = torch.zeros(1, 3, 4, device="cuda")
    with pytest.raises(binding.MesaError):  # 2 does not divide 3
        binding.mesa_delta_forward_chunked(q, q, v, g, g)
    with pytest.raises(binding.MesaError):  # gates of another shape
        binding.mesa_delta_forward_chunked(q, q, q, g, g)
    with pytest.raises(binding.MesaError):  # not contiguous
        binding.mesa_delta_forward_chunked(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, g[:, :2].contiguous(),
                                           g[:, :2].contiguous())


def test_wait_give_up_reports_timeout_and_the_next_call_is_clean():
    """The tensor-core kernels' bounded waits made to give up at once: a status, no hang."""
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(19, "bf16", 1, 2, 2, 300, 128, 128, "open")
    t = upload(s, "bf16")
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    sizes = (1, 2, 2, 300, 128, 128, torch.bfloat16)
    wf = torch.empty(binding.mesa_delta_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    wb = torch.empty(binding.mesa_delta_backward_workspace_size(*sizes), dtype=torch.uint8, device="cuda")

    def run():
        out = binding.mesa_delta_forward_chunked(*args, workspace=wf)
        grads = binding.mesa_delta_backward_chunked(*args, t["dout"], workspace=wb)
        return [out, *grads], [binding.mesa_forward_status_code(w) for w in (wf, wb)]

    want, codes = run()
    assert codes == [(binding.MESA_OK, 0)] * 2
    binding.mesa_debug_set_wait_limit(0)
    try:
        _, codes = run()
    finally:
        binding.mesa_debug_set_wait_limit(-1)
    assert codes[0][0] == binding.MESA_ERR_TIMEOUT and codes[0][1] & 1 and not codes[0][1] & 4, codes
    got, codes = run()
    assert codes == [(binding.MESA_OK, 0)] * 2
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def _long_inputs(T, gates, S0, seed=31):
    """One (batch, head) unit pair of T tokens, bf16, d = 128: so few units that the sequence is cut
    into segments."""
    s = ref.rule_inputs(seed, "bf16", 1, 2, 2, T, 128, 128, "open", S0)
    r = np.random.default_rng(seed + 1)
    if gates == "kept":  # hardly any decay: every segment needs the state before it
        s["gamma"] = r.uniform(0.9995, 1.0, s["gamma"].shape).astype(np.float32)
    elif gates == "loud":  # the first half 2^30 times louder than the rest: still there after a long decay
        s["v"][:, :, :T // 2] *= 2.0 ** 15
        s["v"][:, :, T // 2:] *= 2.0 ** -15
        s["gamma"] = r.uniform(0.97, 1.0, s["gamma"].shape).astype(np.float32)
    elif gates == "mixed":  # one unit that keeps, one that forgets; a closed gate and zero betas
        s["gamma"][:, 0] = r.uniform(0.999, 1.0, s["gamma"][:, 0].shape).astype(np.float32)
        s["gamma"][:, 1, T // 3] = 0.0
        s["beta"][:, :, T - T // 5:] = 0.0
    return s


LONG = [(1921, "open", True), (2500, "kept", True), (2048, "loud", False), (3001, "mixed", True), (2111, "kept", False)]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_sequences_of_few_units(case):
    import torch

    from mesa_layer_gb300 import binding
    T, gates, S0 = case
    s = _long_inputs(T, gates, S0)
    t = upload(s, "bf16")
    SF = torch.full((1, 2, 128, 128), float("nan"), device="cuda")
    out = binding.mesa_delta_forward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], SCALE, S0=t["S0"], S_final=SF)
    o, S = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["S0"])
    if gates == "loud":  # (token norms span 2^30: by parts)
        parts = [slice(i, i + 64) for i in range(0, T, 64)]
        assert max(err(out[:, :, p], o[:, :, p]) for p in parts) <= TOL["bf16"]
    assert err(out, o) <= TOL["bf16"]
    assert err(SF, S) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("case", LONG[:2] + LONG[3:], ids=str)
def test_gradients_of_long_sequences_of_few_units(case):
    import torch

    from mesa_layer_gb300 import binding
    T, gates, S0 = case
    s = _long_inputs(T, gates, S0)
    t = upload(s, "bf16")
    dS0 = torch.full((1, 2, 128, 128), float("nan"), device="cuda") if S0 else None
    got = dict(zip(("dq", "dk", "dv", "dgamma", "dbeta"), binding.mesa_delta_backward_chunked(
        t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE, S0=t["S0"], dS_final=t["dS_final"], dS0=dS0)))
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    found = {n: err(x, want[n]) for n, x in got.items()}
    assert max(found.values()) <= TOL["bf16"], found
    if S0:
        assert err(dS0, want["dS0"]) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("what", ["v", "beta", "S0"])
def test_nonfinite_values_last_through_long_sequences(what):
    """A NaN early in a long sequence is still in the state at its end (0.9 ^ 3000 of it)."""
    import torch

    from mesa_layer_gb300 import binding
    s = _long_inputs(3000 + 1, "open", True)
    t = upload(s, "bf16")
    if what == "S0":
        t["S0"][0, 1, 5, 7] = float("nan")
    elif what == "v":
        t["v"][0, 1, 70, 5] = float("inf")
    else:
        t["beta"][0, 1, 70] = float("nan")
    SF = torch.zeros((1, 2, 128, 128), device="cuda")
    ws = torch.empty(binding.mesa_delta_workspace_size(1, 2, 2, 3001, 128, 128, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    out = binding.mesa_delta_forward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], SCALE, S0=t["S0"], S_final=SF,
                                             workspace=ws)
    assert binding.mesa_forward_status(ws) != 0
    assert torch.isfinite(SF[0, 0]).all() and torch.isfinite(out[0, 0]).all()
    assert not torch.isfinite(SF[0, 1, 5]).any()
    assert not torch.isfinite(out[0, 1, -1, 5])


@pytest.mark.parametrize("dtype,d,T", [("f32", 64, 100), ("f32", 64, 1500), ("bf16", 128, 100), ("bf16", 128, 2500)])
def test_final_states_may_replace_the_first(dtype, d, T):
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(41, dtype, 1, 2, 1, T, d, d, "open", True)
    t = upload(s, dtype)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    S, A = torch.empty_like(t["S0"]), torch.empty_like(t["S0"])
    out = binding.mesa_delta_forward_chunked(*args, S0=t["S0"], S_final=S)
    grads = binding.mesa_delta_backward_chunked(*args, t["dout"], S0=t["S0"], dS_final=t["dS_final"], dS0=A)
    S2, A2 = t["S0"].clone(), t["dS_final"].clone()
    assert torch.equal(binding.mesa_delta_forward_chunked(*args, S0=S2, S_final=S2), out) and torch.equal(S2, S)
    again = binding.mesa_delta_backward_chunked(*args, t["dout"], S0=t["S0"], dS_final=A2, dS0=A2)
    assert torch.equal(A2, A) and all(torch.equal(x, y) for x, y in zip(again, grads))


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_long_sequences_write_inside_their_buffers_and_repeat(dtype, d):
    import torch

    from mesa_layer_gb300 import binding
    from test_gpu_canary import Guarded, workspace
    T = 2345
    s = ref.rule_inputs(42, dtype, 1, 2, 2, T, d, d, "packed", True)
    t = upload(s, dtype)
    td = t["q"].dtype
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    wf = workspace(binding.mesa_delta_workspace_size(1, 2, 2, T, d, d, td))
    wb = workspace(binding.mesa_delta_backward_workspace_size(1, 2, 2, T, d, d, td))
    runs = []
    for _ in range(2):
        out, SF, dS0 = Guarded((1, 2, T, d), td), Guarded((1, 2, d, d), torch.float32), Guarded((1, 2, d, d), torch.float32)
        g = [Guarded((1, 2, T, d), td) for _ in range(3)] + [Guarded((1, 2, T), td) for _ in range(2)]
        binding.mesa_delta_forward_chunked(*args, out=out.t, S0=t["S0"], S_final=SF.t, workspace=wf.t)
        binding.mesa_delta_backward_chunked(*args, t["dout"], 1.0, t["S0"], t["dS_final"], *(x.t for x in g), dS0=dS0.t,
                                            workspace=wb.t)
        assert all(x.intact() for x in (out, SF, dS0, wf, wb, *g))
        runs.append([x.t for x in (out, SF, dS0, *g)])
    assert all(torch.equal(x, y) for x, y in zip(*runs))


def test_wait_give_up_in_a_long_sequence_reports_timeout():
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(43, "bf16", 1, 1, 1, 2100, 128, 128, "open")
    t = upload(s, "bf16")
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    ws = torch.empty(binding.mesa_delta_workspace_size(1, 1, 1, 2100, 128, 128, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    want = binding.mesa_delta_forward_chunked(*args, workspace=ws)
    assert binding.mesa_forward_status(ws) == 0
    binding.mesa_debug_set_wait_limit(0)
    try:
        binding.mesa_delta_forward_chunked(*args, workspace=ws)
        code, bits = binding.mesa_forward_status_code(ws)
    finally:
        binding.mesa_debug_set_wait_limit(-1)
    assert code == binding.MESA_ERR_TIMEOUT and bits & 1 and not bits & 4
    assert torch.equal(binding.mesa_delta_forward_chunked(*args, workspace=ws), want)
    assert binding.mesa_forward_status(ws) == 0


def test_gradients_across_a_long_sequence_with_loud_ends():
    """dL/dout 2^30 times louder in the second half: it still rules the gradients of the first half
    long before it (0.985 ^ 1000 = 2^-22 of it), compared chunk by chunk."""
    import torch

    from mesa_layer_gb300 import binding
    T = 2048
    s = _long_inputs(T, "open", True, 51)
    s["gamma"] = np.random.default_rng(52).uniform(0.97, 1.0, s["gamma"].shape).astype(np.float32)
    s["dout"][:, :, T // 2:] *= 2.0 ** 15
    s["dout"][:, :, :T // 2] *= 2.0 ** -15
    t = upload(s, "bf16")
    dS0 = torch.full((1, 2, 128, 128), float("nan"), device="cuda")
    got = dict(zip(("dq", "dk", "dv", "dgamma", "dbeta"), binding.mesa_delta_backward_chunked(
        t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE, S0=t["S0"], dS_final=t["dS_final"], dS0=dS0)))
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    for n in ("dq", "dk", "dv"):
        for i in range(0, T, 64):
            assert err(got[n][:, :, i:i + 64], want[n][:, :, i:i + 64]) <= TOL["bf16"], (n, i)
    assert err(dS0, want["dS0"]) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("what", ["dout", "dS_final"])
def test_nonfinite_gradients_last_through_long_sequences(what):
    """A NaN late in a long sequence reaches the first token's gradients (0.9 ^ 3000 of it)."""
    import torch

    from mesa_layer_gb300 import binding
    t = upload(_long_inputs(3001, "open", True), "bf16")
    if what == "dout":
        t["dout"][0, 1, 2950, 5] = float("nan")
    else:
        t["dS_final"][0, 1, 5, 7] = float("inf")
    dS0 = torch.zeros((1, 2, 128, 128), device="cuda")
    dv = binding.mesa_delta_backward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE, S0=t["S0"],
                                             dS_final=t["dS_final"], dS0=dS0)[2]
    assert torch.isfinite(dS0[0, 0]).all() and torch.isfinite(dv[0, 0]).all()
    assert not torch.isfinite(dS0[0, 1, 5]).any() and not torch.isfinite(dv[0, 1, 0, 5])
