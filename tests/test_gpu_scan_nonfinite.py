"""What is not finite in one token of the scan reaches what depends on it by the recurrence, and nothing else: outputs and
gradients on the other side of it are those of clean inputs, bit for bit (documents in a row apart: those share what is not
finite, as the header says)."""
import pytest
import torch

from test_gpu_ssm import BF16, F32, forward, lib, make  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu
SIZES = [(F32, 32, 32), (F32, 128, 64), (F32, 64, 128), (BF16, 128, 128), (BF16, 128, 64), (BF16, 64, 64), (BF16, 32, 128)]
TOKENS = [0, 1, 31, 40, 64, 127, 128, 190, 298, 299]
T, B, H, Hk = 300, 1, 4, 2


def same(x, y):
    return torch.equal(x, y)


def case(dtype, dk, dv, states=True):
    return make(dtype, B, H, Hk, T, dk, dv, seed=17, states=states, steps=(1e-3, 1e-1))


@pytest.mark.parametrize("bad", [torch.inf, -torch.inf, torch.nan])
@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_forward(lib, dtype, dk, dv, bad):  # noqa: F811
    clean = case(dtype, dk, dv)
    out, S = forward(lib, clean)
    for i, t in enumerate(TOKENS):
        h, p, n = i % H, (37 * i + 5) % dv, (29 * i + 3) % dk
        s = dict(clean, v=clean["v"].clone())
        s["v"][0, h, t, p] = bad
        o, E = forward(lib, s)
        others = torch.arange(dv, device="cuda") != p
        assert not o[0, h, t:, p].isfinite().any() and same(o[0, h, :t, p], out[0, h, :t, p]), t
        assert same(o[0, h][:, others], out[0, h][:, others]) and not E[0, h, p].isfinite().any() and same(E[0, h, others], S[0, h, others])
        rest = torch.arange(H, device="cuda") != h
        assert same(o[:, rest], out[:, rest]) and same(E[:, rest], S[:, rest])
        g = h // (H // Hk)
        mine = torch.arange(H, device="cuda") // (H // Hk) == g
        s = dict(clean, k=clean["k"].clone())
        s["k"][0, g, t, n] = bad
        o, E = forward(lib, s)
        assert not o[0, mine, t:].isfinite().any() and same(o[:, :, :t], out[:, :, :t]) and same(o[:, ~mine], out[:, ~mine])
        assert not E[0, mine][:, :, n].isfinite().any()
        s = dict(clean, q=clean["q"].clone())
        s["q"][0, g, t, n] = bad
        o, E = forward(lib, s)
        keep = torch.arange(T, device="cuda") != t
        assert not o[0, mine, t].isfinite().any() and same(o[:, :, keep], out[:, :, keep]) and same(E, S)
        s = dict(clean, dt=clean["dt"].clone())
        s["dt"][0, h, t] = bad if bad != -torch.inf else torch.nan  # (-infinity is padding)
        o, E = forward(lib, s)
        assert not o[0, h, t].isfinite().any() and same(o[0, h, :t], out[0, h, :t]) and same(o[:, rest], out[:, rest])


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_forward_with_several_of_them(lib, dtype, dk, dv):  # noqa: F811
    """Each channel from its own first one on."""
    clean = case(dtype, dk, dv)
    out, S = forward(lib, clean)
    g = torch.Generator().manual_seed(3)
    at = torch.rand(B, H, T, dv, generator=g).cuda() < 2e-3
    s = dict(clean, v=torch.where(at, torch.nan, clean["v"].float()).to(dtype))
    o, E = forward(lib, s)
    gone = at.cumsum(2) > 0
    assert gone.any() and not gone.all() and torch.equal(o.isnan(), gone) and same(o[~gone], out[~gone])
    assert torch.equal(E.isnan().all(-1), gone[:, :, -1]) and same(E[~gone[:, :, -1]], S[~gone[:, :, -1]])


@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_forward_with_states_in_place(lib, dtype, dk, dv):  # noqa: F811
    """S_final over S0's memory, captured and replayed: a walk done over begins from the same state."""
    clean = case(dtype, dk, dv)
    out, S = forward(lib, clean)
    v, state, o = clean["v"].clone(), clean["S0"].clone(), torch.empty_like(out)
    scan = (clean["q"], clean["k"], v, clean["dt"], clean["A"])

    def call():
        lib.mesa_ssm_forward_chunked(*scan, dt_bias=clean["dt_bias"], skip=clean["skip"], out=o, S0=state, S_final=state)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    others = torch.arange(dv, device="cuda") != 3
    for bad in (torch.nan, 1.0, -torch.inf):
        v.copy_(clean["v"])
        v[0, 1, 140, 3] = bad
        state.copy_(clean["S0"])
        graph.replay()
        torch.cuda.synchronize()
        assert same(o[:, 1, :, others], out[:, 1, :, others]) and same(o[:, 1, :140], out[:, 1, :140]) and same(state[:, 1, others], S[:, 1, others])
        assert same(o[:, [0, 2, 3]], out[:, [0, 2, 3]]) and same(state[:, [0, 2, 3]], S[:, [0, 2, 3]])
        assert bool(o[0, 1, 140:, 3].isfinite().all() if bad == 1.0 else not o[0, 1, 140:, 3].isfinite().any())
        assert bool(state[0, 1, 3].isfinite().all() if bad == 1.0 else not state[0, 1, 3].isfinite().any())


def test_forward_in_segments(lib):  # noqa: F811
    """Few long units: a segment's first walk carries it, the second keeps what came before."""
    for dk, dv in ((128, 128), (128, 64), (64, 64)):
        s = make(BF16, 1, 16, 16, 20 * 128 - 3, dk, dv, seed=2, states=True, steps=(1e-3, 1e-2))
        out, S = forward(lib, s)
        for t in (100, 777, 1300, 2400, 2556):
            x = dict(s, v=s["v"].clone())
            x["v"][0, 5, t, 7] = torch.nan
            o, E = forward(lib, x)
            gone = torch.zeros_like(out, dtype=torch.bool)
            gone[0, 5, t:, 7] = True
            assert torch.equal(o.isnan(), gone) and same(o[~gone], out[~gone]) and E[0, 5, 7].isnan().all()


def backward(lib, s):  # noqa: F811
    return dict(zip(("q", "k", "v", "dt"), lib.mesa_ssm_backward_chunked(
        s["q"], s["k"], s["v"], s["dt"], s["A"], s["dout"], dt_bias=s["dt_bias"], skip=s["skip"], S0=s["S0"], dS_final=s["dS_final"],
        gates_dtype=F32)[:4]))


@pytest.mark.parametrize("own", [False, True])  # (query and key heads of their own: written without a sum over heads)
@pytest.mark.parametrize("bad", [torch.inf, torch.nan])
@pytest.mark.parametrize("dtype,dk,dv", SIZES)
def test_backward(lib, dtype, dk, dv, bad, own):  # noqa: F811
    clean = make(dtype, B, H, H if own else Hk, T, dk, dv, seed=18, states=True, steps=(1e-3, 1e-1))
    want = backward(lib, clean)
    at = torch.arange(T, device="cuda")
    for i, t in enumerate(TOKENS):
        before, after, elsewhere = at < t, at > t, at != t
        for name in ("q", "k", "v", "dout"):
            x = clean[name].clone()
            c = (31 * i + 7) % x.shape[-1]
            h = i % x.shape[1]
            x[0, h, t, c] = bad
            got = backward(lib, dict(clean, **{name: x}))
            shared = name in "qk" and not own
            value = slice(2 * h, 2 * h + 2) if shared else slice(h, h + 1)  # the value heads that take part
            key = h if own or shared else h // 2
            for n, y in got.items():  # other heads
                rest = torch.ones(y.shape[1], dtype=torch.bool, device="cuda")
                rest[key if n in "qk" else value] = False
                assert same(y[:, rest], want[n][:, rest]), (name, t, n)
            same_at = {  # tokens whose gradients do not see it
                "q": dict(q=elsewhere, k=after, v=after, dt=after), "k": dict(q=before, k=at >= 0, v=elsewhere, dt=before),
                "v": dict(q=before, k=elsewhere, v=at >= 0, dt=before), "dout": dict(q=elsewhere, k=after, v=after, dt=after)}[name]
            for n, keep in same_at.items():
                if name == "q" and n == "q":  # dq does not depend on q at all
                    keep = at >= 0
                assert same(got[n][:, :, keep], want[n][:, :, keep]), (name, t, n)
            # and what does is not finite
            if name == "k":
                assert not got["q"][0, key, t:, c].isfinite().any() and not got["v"][0, value, t].isfinite().any()
            if name == "q":
                assert not got["k"][0, key, :t + 1, c].isfinite().any() and not got["v"][0, value, :t + 1].isfinite().any()
            if name == "v":
                assert not got["q"][0, key, t:].isfinite().any() and not got["k"][0, key, t].isfinite().any()
            if name == "dout":
                others = torch.arange(dv, device="cuda") != c
                assert same(got["v"][0, :, :, others], want["v"][0, :, :, others])
                assert not got["q"][0, key, t].isfinite().any() and not got["k"][0, key, :t + 1].isfinite().any()
                assert not got["v"][0, value, :t + 1, c].isfinite().any()
        x = clean["dt"].clone()
        h = i % H
        x[0, h, t] = bad
        got = backward(lib, dict(clean, dt=x))
        key = h if own else h // 2
        rest = torch.arange(H, device="cuda") != h
        assert same(got["q"][0, key, :t], want["q"][0, key, :t]) and not got["k"][0, key, t].isfinite().any()
        assert same(got["v"][:, rest], want["v"][:, rest]) and same(got["dt"][:, rest], want["dt"][:, rest])
