"""Scan, convolution and norm with rotation: backward passes and steps captured in a graph and replayed with other
inputs; two calls at once on streams of their own; long sequences in segments, with what is not finite in them."""
import pytest
import torch

from test_gpu_ssm import BF16, F32, STATE_TOL, TOL, lib, make, off  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def captured(call):
    """The graph of call(), warmed up on a side stream; its outputs are call()'s own buffers."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def refill(tensors, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in tensors:
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))


def ssm_backward(lib, s, **kw):
    return lib.mesa_ssm_backward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"],
                                         starts=s["starts"], S0=s["S0"], dS_final=s["dS_final"], gates_dtype=F32, **kw)


@pytest.mark.parametrize("dtype,T,dk,dv", [(F32, 300, 64, 64), (BF16, 300, 128, 128), (BF16, 2500, 128, 64), (BF16, 300, 64, 64)])
def test_scan_backward_captured(lib, dtype, T, dk, dv):  # noqa: F811 (2500 tokens of few units: in segments)
    s = make(dtype, 1, 2, 1, T, dk, dv, seed=T, packed=True, states=True)
    dS0 = torch.empty_like(s["S0"])
    graph, out = captured(lambda: ssm_backward(lib, s, dS0=dS0))
    for seed in (1, 2):
        refill((s["q"], s["k"], s["v"], s["dout"], s["S0"], s["dS_final"]), seed)
        s["q"].mul_(dk ** -0.5)
        graph.replay()
        got = [t.clone() for t in (*out, dS0)]
        want = (*ssm_backward(lib, s, dS0=dS0), dS0)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF16, 128)])
def test_scan_step_captured(lib, dtype, d):  # noqa: F811
    s = make(dtype, 3, 4, 2, 1, d, d, seed=5, states=True)
    row = [s[n][:, :, 0].contiguous() for n in ("q", "k", "v", "dt")]
    state, other = s["S0"].clone(), s["S0"].clone()

    def call(S):
        return lib.mesa_ssm_step(S, *row, s["A"], dt_bias=s["dt_bias"], skip=s["skip"])

    graph, out = captured(lambda: call(state))
    state.copy_(other)
    for seed in range(3):
        refill(row, seed)
        graph.replay()
        assert torch.equal(out, call(other)) and torch.equal(state, other)


def test_convolution_and_rotation_backward_captured(lib):  # noqa: F811
    B, H, T, d = 2, 3, 131, 64
    x, dout, q, k, dq, dk = (torch.empty(B, H, T, d, device="cuda", dtype=BF16) for _ in range(6))
    w, bias, wq, inv = (torch.rand(n, device="cuda") + 0.5 for n in ((H, d, 4), (H, d), (d,), (d // 2,)))
    starts = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    starts[:, 40] = True
    positions = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)

    def call():
        return (*lib.mesa_causal_conv_backward(x, w, dout, bias, starts=starts),
                *lib.mesa_qk_norm_rotary_backward(q, k, dq, dk, wq, wq, inv, positions))

    refill((x, dout, q, k, dq, dk), 0)
    graph, out = captured(call)
    for seed in (1, 2):
        refill((x, dout, q, k, dq, dk), seed)
        starts.copy_(starts.roll(17 * seed, 1))
        positions.add_(1000)
        graph.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


@pytest.mark.parametrize("T", [300, 2500])
def test_two_scans_at_once(lib, T):  # noqa: F811
    """Calls of two streams, each with memory of its own, and with sums of their own."""
    calls = [make(BF16, 2, 4, 2, T, 128, 128, seed=n, packed=n == 1, states=True) for n in range(2)]
    want = [ssm_backward(lib, s) for s in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = [ssm_backward(lib, s, stream=st) for s, st in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


def chunked(s, L=64):
    """out, S_final of one unit's scan in 64 bits, L tokens at once."""
    q, k, v, dt = (s[n][0, 0].double() for n in ("q", "k", "v", "dt"))
    step = torch.nn.functional.softplus(dt + s["dt_bias"].double())
    log = step * s["A"].double()
    S, out = s["S0"][0, 0].double(), torch.empty_like(v)
    for t in range(0, len(q), L):
        e = slice(t, t + L)
        c = log[e].cumsum(0)
        M = torch.exp((c[:, None] - c[None]).tril()).tril() * step[e]
        out[e] = c.exp()[:, None] * (q[e] @ S.T) + (M * (q[e] @ k[e].T)) @ v[e] + s["skip"].double() * v[e]
        S = c[-1].exp() * S + (v[e] * ((c[-1] - c).exp() * step[e])[:, None]).T @ k[e]
    return out, S


@pytest.mark.parametrize("steps", [(1e-6, 2e-6), (1e-4, 2e-4), (1e-2, 2e-2), (0.5, 1.0)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 64)])
def test_segments(lib, dk, dv, steps):  # noqa: F811
    """One long unit (64 chunks, in segments), heads that forget nothing to all: what each segment leaves is weighed by
    the decay after it."""
    s = make(BF16, 1, 1, 1, 64 * 128 - 3, dk, dv, seed=7, states=True, steps=steps)
    S = torch.empty_like(s["S0"])
    out = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"], S0=s["S0"], S_final=S)
    want, want_S = chunked(s)
    assert off(out[0, 0], want) <= TOL[BF16] and off(S[0, 0], want_S) <= STATE_TOL[BF16]


@pytest.mark.parametrize("steps", [(1e-4, 2e-4), (0.5, 1.0)])
@pytest.mark.parametrize("bad", [torch.nan, torch.inf])
def test_not_finite_stays_over_the_segments(lib, bad, steps):  # noqa: F811
    """What is not finite reaches every later token's output, and every earlier token's gradient of v."""
    T, d = 64 * 128 - 3, 128
    s = make(BF16, 1, 1, 1, T, d, d, seed=8, steps=steps)
    S = torch.empty(1, 1, d, d, device="cuda")
    s["v"][0, 0, 130, 3] = bad
    out = lib.mesa_ssm_forward_chunked(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], skip=s["skip"], S_final=S)
    gone = ~out[0, 0].isfinite()
    assert gone[130:, 3].all() and not gone[:, :3].any() and not gone[:, 4:].any() and not gone[:128].any()
    assert not S[0, 0, 3].isfinite().any() and S[0, 0, 4:].isfinite().all()
    s["v"][0, 0, 130, 3] = 1.0
    s["dout"][0, 0, T - 200, 3] = bad
    dv = ssm_backward(lib, s)[2][0, 0]
    gone = ~dv.isfinite()
    assert gone[:T - 199, 3].all() and not gone[:, :3].any() and not gone[:, 4:].any() and not gone[63 * 128:].any()
