"""The gated delta rule on the GPU where inputs are unusual: chunks without queries, gates above one,
correlated keys, non-finite values, other streams.  Against the 64-bit restatement with the tolerances of
test_gpu_delta.py, whose derivation does not depend on the inputs, unless a test says otherwise."""
import numpy as np
import pytest

import delta_reference as ref
from test_gpu_delta import SCALE, STATE_TOL, TOL, err, upload

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dgamma", "dbeta")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mesa_layer_gb300 import binding, build
    build.build()
    binding.load()


def sizes(t):
    B, H, T, dv = t["v"].shape
    return B, H, t["q"].shape[1], T, t["q"].shape[-1], dv, t["q"].dtype


def forward(t):
    """out, S_final, (status code, flags)."""
    import torch

    from mesa_layer_gb300 import binding
    B, H, Hk, T, dk, dv, td = sizes(t)
    SF = torch.full((B, H, dv, dk), float("nan"), device="cuda")
    ws = torch.empty(binding.mesa_delta_workspace_size(*sizes(t)), dtype=torch.uint8, device="cuda")
    out = binding.mesa_delta_forward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], SCALE, S0=t["S0"], S_final=SF,
                                             workspace=ws)
    return out, SF, binding.mesa_forward_status_code(ws)


def backward(t):
    """The gradients by name (dS0 among them), (status code, flags)."""
    import torch

    from mesa_layer_gb300 import binding
    B, H, Hk, T, dk, dv, td = sizes(t)
    dS0 = torch.full((B, H, dv, dk), float("nan"), device="cuda")
    ws = torch.empty(binding.mesa_delta_backward_workspace_size(*sizes(t)), dtype=torch.uint8, device="cuda")
    got = binding.mesa_delta_backward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], SCALE, S0=t["S0"],
                                              dS_final=t["dS_final"], dS0=dS0, workspace=ws)
    return dict(zip((*GRADS, "dS0"), (*got, dS0))), binding.mesa_forward_status_code(ws)


def check_forward(s, dtype):
    out, SF, status = forward(upload(s, dtype))
    assert status == (0, 0)
    o, S = ref.rule_forward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["S0"])
    found = {"out": err(out, o), "S_final": err(SF, S)}
    assert found["out"] <= TOL[dtype] and found["S_final"] <= STATE_TOL[dtype], found


def check_backward(s, dtype):
    got, status = backward(upload(s, dtype))
    assert status == (0, 0)
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    found = {n: err(x, want[n]) for n, x in got.items()}
    assert max(found[n] for n in GRADS) <= TOL[dtype] and found["dS0"] <= STATE_TOL[dtype], found


@pytest.mark.parametrize("what", ["no queries", "no queries, loud gradients", "padding without queries", "faint queries",
                                  "no queries anywhere", "no keys"])
def test_gradients_of_chunks_without_queries(what):
    """The second 64-token chunk (of three) has no queries, or far smaller ones than its keys; as padding it
    writes nothing and is not read either."""
    s = ref.rule_inputs(61, "bf16", 1, 2, 1, 150, 128, 128, "open", True)
    mid = slice(64, 128)
    if what == "no queries":
        s["q"][:, :, mid] = 0.0
    elif what == "no queries, loud gradients":
        s["q"][:, :, mid] = 0.0
        for n in ("dout", "dS_final"):
            s[n] *= 2.0 ** 12
    elif what == "padding without queries":  # the last chunk
        for n in ("q", "beta", "dout"):
            s[n][:, :, 128:] = 0.0
        s["dS_final"][:] = 0.0
    elif what == "faint queries":
        s["q"][:, :, mid] *= 2.0 ** -60
        s["dout"] *= 2.0 ** 12
    elif what == "no queries anywhere":
        s["q"][:] = 0.0
    else:
        s["k"][:, :, mid] = 0.0
    got, status = backward(upload(s, "bf16"))
    assert status == (0, 0)
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    for n in GRADS:  # chunk by chunk
        for i in range(0, 150, 64):
            assert err(got[n][:, :, i:i + 64], want[n][:, :, i:i + 64]) <= TOL["bf16"], (n, i)
    assert err(got["dS0"], want["dS0"]) <= STATE_TOL["bf16"]


@pytest.mark.parametrize("T", [16, 17, 64, 130, 300])
@pytest.mark.parametrize("gates", [(1.0, 1.03), (1.03, 1.03), (1.0, 1.05), (0.9, 1.1), (1.09, 1.09)], ids=str)
def test_gates_above_one(T, gates):
    """A state that grows: the same on both sides of the 16 tokens from which chunks are taken."""
    s = ref.rule_inputs(62, "bf16", 1, 2, 2, T, 128, 128, "open", True)
    s["gamma"] = np.random.default_rng(63).uniform(*gates, s["gamma"].shape).astype(np.float32)
    check_forward(s, "bf16")
    check_backward(s, "bf16")


@pytest.mark.parametrize("T", [16, 17, 64, 130, 300])
def test_a_burst_of_gates_is_reported_by_the_chunked_form(T):
    """1.5^24 = 2^14 in a chunk is more than its fp16 operands hold beside the decays: reported, not rounded
    away.  (Up to 16 tokens the forward is a recurrence, which takes any gate.)"""
    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(62, "bf16", 1, 2, 2, T, 128, 128, "open", True)
    s["gamma"][:] = 1.5
    s["gamma"][:, :, 24:] = 0.95
    if T <= 16:
        check_forward(s, "bf16")
    else:
        out, SF, status = forward(upload(s, "bf16"))
        assert status == (binding.MESA_ERR_NONFINITE, 2)
        assert not out.isfinite().any() and not SF.isfinite().any()
    got, status = backward(upload(s, "bf16"))
    assert status == (binding.MESA_ERR_NONFINITE, 2)
    assert not got["dS0"].isfinite().any() and not got["dk"][:, :, :64].isfinite().any()


def test_negative_gates_are_reported_by_the_chunked_form():
    """Chunks take decays as logarithms: a gate below zero has none."""
    t = upload(ref.rule_inputs(64, "bf16", 1, 2, 2, 100, 128, 128, "open", True), "bf16")
    t["gamma"][0, 1, 70] = -0.5
    from mesa_layer_gb300 import binding
    out, _, status = forward(t)
    assert status == (binding.MESA_ERR_NONFINITE, 2)
    assert out[0, 0].isfinite().all() and not out[0, 1, 70:].isfinite().any()
    got, status = backward(t)
    assert status == (binding.MESA_ERR_NONFINITE, 2)
    assert got["dv"][0, 0].isfinite().all()


@pytest.mark.parametrize("dtype,dk,dv,Hk,T", [("f32", 64, 64, 2, 70), ("f32", 16, 32, 1, 200), ("bf16", 64, 64, 1, 90),
                                              ("bf16", 32, 128, 2, 5), ("f32", 32, 16, 1, 900), ("bf16", 128, 128, 2, 70)],
                         ids=str)
@pytest.mark.parametrize("what", ["dout", "beta", "dS_final", "overflow"])
def test_nonfinite_gradients_are_reported(dtype, dk, dv, Hk, T, what):
    from mesa_layer_gb300 import binding
    t = upload(ref.rule_inputs(65, dtype, 1, 2, Hk, T, dk, dv, "open", True), dtype)
    assert backward(t)[1] == (binding.MESA_OK, 0)
    if what == "dout":
        t["dout"][0, 1, T // 2, 3] = float("nan")
    elif what == "beta":
        t["beta"][0, 1, T // 2] = float("inf")
    elif what == "dS_final":
        t["dS_final"][0, 1, 5, 7] = float("nan")
    else:  # finite inputs, a sum that is not
        t["dS_final"][0, 1] = 3e38
    got, status = backward(t)
    assert status == (binding.MESA_ERR_NONFINITE, 2)
    assert got["dv"][0, 0].isfinite().all() and not got["dv"][0, 1].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_whose_sum_over_heads_overflows_are_reported(dtype):
    """Two value heads share a key head; each part of dq is below the largest fp32 value, their sum is not."""
    import torch

    from mesa_layer_gb300 import binding
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    t = {n: torch.zeros(1, h, 1, 32, device="cuda", dtype=td) for n, h in (("q", 1), ("k", 1), ("v", 2), ("dout", 2))}
    t["k"][..., 0] = 1.0  # S = v k^T, dq = S^T dout = k (v . dout)
    t["v"][..., 0] = 2.0 ** 63
    t["dout"][..., 0] = 2.0 ** 64
    t.update(gamma=torch.ones(1, 2, 1, device="cuda"), beta=torch.ones(1, 2, 1, device="cuda"), S0=None, dS_final=None)
    ws = torch.empty(binding.mesa_delta_backward_workspace_size(*sizes(t)), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        dq = binding.mesa_delta_backward_chunked(t["q"], t["k"], t["v"], t["gamma"], t["beta"], t["dout"], workspace=ws)[0]
        status = binding.mesa_forward_status_code(ws)
        if t["v"][0, 1, 0, 0] == 0:
            break
        assert status == (binding.MESA_ERR_NONFINITE, 2) and dq[0, 0, 0, 0].isinf()
        t["v"][0, 1] = 0.0
    assert status == (binding.MESA_OK, 0) and dq[0, 0, 0, 0] == 2.0 ** 127


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 16)])
def test_a_step_reports_its_nonfinite_outputs(dtype, d):
    from mesa_layer_gb300 import binding
    t = upload(ref.rule_inputs(66, dtype, 3, 2, 1, 1, d, d, "open", True), dtype)
    args = [t[n][:, :, 0].contiguous() for n in ("q", "k", "v", "gamma", "beta")]
    binding.mesa_decode_status()  # clear
    clean = binding.mesa_delta_step(t["S0"].clone(), *args)
    assert binding.mesa_decode_status() == (binding.MESA_OK, 0)
    args[2][1, 0, 3] = float("inf")
    out = binding.mesa_delta_step(t["S0"].clone(), *args)
    assert binding.mesa_decode_status() == (binding.MESA_ERR_NONFINITE, 2)
    assert not out[1, 0, 3].isfinite()
    out[1, 0, 3] = clean[1, 0, 3]
    assert out.equal(clean)
    assert binding.mesa_decode_status() == (binding.MESA_OK, 0)


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_another_stream_leaves_freed_blocks_of_this_one_alone(dtype, d):
    """Blocks of the outputs' sizes freed here while work that writes them is still queued: a call on
    another stream in the meantime takes other memory."""
    import torch

    from mesa_layer_gb300 import binding
    t = upload(ref.rule_inputs(75, dtype, 1, 4, 2, 300, d, d, "open"), dtype)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    y, w = t["v"].reshape(-1, d), torch.ones(d, device="cuda")

    def calls(stream=None):
        return [binding.mesa_delta_forward_chunked(*args, stream=stream),
                *binding.mesa_delta_backward_chunked(*args, t["dout"], stream=stream),
                *binding.mesa_block_norm(y, y, w_post=w, w_pre=w, stream=stream),
                *(x for x in binding.mesa_block_norm_backward(y, y, y, dh=y, w_post=w, w_pre=w, stream=stream)
                  if x is not None)]

    want = calls()
    blocks = [x.nbytes for x in want] + [binding.mesa_delta_workspace_size(*sizes(t)),
                                         binding.mesa_delta_backward_workspace_size(*sizes(t))]
    a = torch.ones(4096, 4096, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):  # milliseconds of work
        b = a @ a
    for n in 2 * blocks:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)  # freed at once, written later
    got = calls(side)
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy  # (else it showed nothing)
    assert all(x.equal(z) for x, z in zip(got, want))


def correlated(seed, T, cosine, betas, queries, S0=True, H=2, Hk=2):
    """Keys (and queries) of a head about a common direction; slow gates."""
    s = ref.rule_inputs(seed, "bf16", 1, H, Hk, T, 128, 128, "open", S0)
    r = np.random.default_rng(seed + 1)

    def unit(x):
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    c = unit(r.standard_normal((1, Hk, 1, 128)))
    for n in ("k", "q") if queries else ("k",):
        s[n] = ref.round_bf16(unit(np.sqrt(cosine) * c + np.sqrt(1.0 - cosine) * unit(s[n])))
    s["beta"] = r.uniform(*betas, s["beta"].shape).astype(np.float32)
    s["gamma"] = r.uniform(0.99, 1.0, s["gamma"].shape).astype(np.float32)
    return s


CORRELATED = [(0.5, (0.0, 1.0), False), (0.9, (0.0, 1.0), True), (0.9, (1.0, 2.0), False)]


@pytest.mark.parametrize("cosine,betas,queries", CORRELATED, ids=str)
def test_correlated_keys(cosine, betas, queries):
    """The triangular factor is far from the identity and the outputs are small sums of large terms."""
    s = correlated(67, 512, cosine, betas, queries)
    check_forward(s, "bf16")
    check_backward(s, "bf16")


@pytest.mark.parametrize("cosine,betas,queries", [*CORRELATED, (0.9, (1.0, 2.0), True)], ids=str)
def test_correlated_keys_in_fp32(cosine, betas, queries):
    """What the header offers where the terms are too large for fp16 operands."""
    s = correlated(67, 512, cosine, betas, queries)
    check_forward(s, "f32")
    check_backward(s, "f32")


@pytest.mark.parametrize("dk,dv,T", [(64, 64, 90), (32, 128, 300), (128, 128, 150)])
def test_gate_gradients_in_fp32(dk, dv, T):
    """What bf16 calls round: on the CUDA cores all the digits of fp32, and rounded the same values."""
    import torch

    from mesa_layer_gb300 import binding
    s = ref.rule_inputs(76, "bf16", 1, 2, 1, T, dk, dv, "packed", True)
    t = upload(s, "bf16")
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta", "dout")]
    states = dict(S0=t["S0"], dS_final=t["dS_final"])
    want = ref.rule_backward(s["q"], s["k"], s["v"], s["gamma"], s["beta"], SCALE, s["dout"], s["S0"], s["dS_final"])
    rounded = binding.mesa_delta_backward_chunked(*args, SCALE, **states)
    mine = torch.full((1, 2, T), float("nan"), device="cuda")
    for options in (dict(gates_dtype=torch.float32), dict(dgamma=mine), dict(dbeta=mine)):
        got = binding.mesa_delta_backward_chunked(*args, SCALE, **states, **options)
        assert got[3].dtype is got[4].dtype is torch.float32
        assert all(x.to(torch.bfloat16).equal(y) for x, y in zip(got, rounded))
        for x, n in zip(got[3:], GRADS[3:]):
            assert err(x, want[n]) <= TOL["bf16" if dk == dv == 128 else "f32"]
    assert mine.isfinite().all()


def test_gate_gradients_of_other_types_are_refused():
    import torch

    from mesa_layer_gb300 import binding
    t = upload(ref.rule_inputs(77, "bf16", 1, 2, 1, 20, 16, 16, "open"), "bf16")
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta", "dout")]
    full = torch.zeros(1, 2, 20, device="cuda")
    for options in (dict(gates_dtype=torch.float64), dict(dgamma=full.half()), dict(dgamma=full, dbeta=full.bfloat16()),
                    dict(dgamma=full, gates_dtype=torch.bfloat16), dict(dbeta=full[:, :1].contiguous())):
        with pytest.raises(binding.MesaError):
            binding.mesa_delta_backward_chunked(*args, **options)
    f = {n: x.float() for n, x in t.items() if x is not None}
    with pytest.raises(binding.MesaError):  # an fp32 call has no bf16 gradients
        binding.mesa_delta_backward_chunked(*(f[n] for n in ("q", "k", "v", "gamma", "beta", "dout")),
                                            gates_dtype=torch.bfloat16)


@pytest.mark.parametrize("H,T", [(2, 300), (1, 2100)])
def test_wait_give_up_of_the_gradients_reports_timeout(H, T):
    """Every tensor-core kernel of the backward (in segments, too) told to give up at its first wait."""
    from mesa_layer_gb300 import binding
    t = upload(ref.rule_inputs(68, "bf16", 1, H, 1, T, 128, 128, "open", True), "bf16")
    want, status = backward(t)
    assert status == (binding.MESA_OK, 0)
    binding.mesa_debug_set_wait_limit(0)
    try:
        _, (code, bits) = backward(t)
    finally:
        binding.mesa_debug_set_wait_limit(-1)
    assert code == binding.MESA_ERR_TIMEOUT and bits & 1 and not bits & 4
    got, status = backward(t)
    assert status == (binding.MESA_OK, 0)
    assert all(got[n].equal(want[n]) for n in want)


@pytest.mark.parametrize("T", [1921, 2500])
def test_long_sequences_with_shared_key_heads(T):
    """Segments of sequences whose value heads share queries and keys."""
    s = ref.rule_inputs(69, "bf16", 1, 4, 2, T, 128, 128, "open", True)
    s["gamma"] = np.random.default_rng(70).uniform(0.998, 1.0, s["gamma"].shape).astype(np.float32)
    check_forward(s, "bf16")
    check_backward(s, "bf16")


@pytest.mark.parametrize("dtype,d,T", [("f32", 32, 150), ("bf16", 128, 150), ("bf16", 128, 2100)])
def test_calls_in_a_graph(dtype, d, T):
    """Every entry point captured into one graph and replayed on other inputs."""
    import torch

    from mesa_layer_gb300 import binding
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    ins = [upload(ref.rule_inputs(71 + i, dtype, 1, 2, 1, T, d, d, "packed", True), dtype) for i in range(2)]
    x = {n: a.clone() for n, a in ins[0].items()}
    y = torch.randn(T, d, device="cuda").to(td)
    w = torch.ones(d, device="cuda")
    S = x["S0"].clone()

    def calls():
        args = [x[n] for n in ("q", "k", "v", "gamma", "beta")]
        out = binding.mesa_delta_forward_chunked(*args, SCALE, S0=x["S0"])
        grads = binding.mesa_delta_backward_chunked(*args, x["dout"], SCALE, S0=x["S0"], dS_final=x["dS_final"])
        o = binding.mesa_delta_step(S, *(a[:, :, 0].contiguous() for a in args))
        h = binding.mesa_block_norm(y, y, w_post=w, w_pre=w)
        n = binding.mesa_block_norm_backward(y, y, y, dh=y, w_post=w, w_pre=w)
        return [out, *grads, o, *h, *(a for a in n if a is not None)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for a in ins[::-1]:
        for n in x:
            x[n].copy_(a[n])
        S.copy_(a["S0"])
        graph.replay()
        got = [c.clone() for c in captured]
        S.copy_(a["S0"])
        assert all(p.equal(q) for p, q in zip(got, calls()))
