"""Cases of the gated delta rule (chunked forward, backward, decode step) and of the block
norm (forward, backward), and their plain forms.

Gated delta rule, per (batch, head) unit, state S [dv, dk], zero (or given) before token 0:
    e_t = v_t - gamma_t S_{t-1} k_t,   u_t = beta_t e_t,
    S_t = gamma_t S_{t-1} + u_t k_t^T,   o_t = scale S_t q_t.
q and k may have fewer heads than v (Hk divides H; head h reads head h // (H / Hk)).

Block norm, per row of D channels (each part optional):
    z = y rsqrt(mean(y^2) + eps) w_post,   x' = x + res_scale silu(gate) z,
    h = x' rsqrt(mean(x'^2) + eps) w_pre.

``own`` false: elementary torch operations in fp32, rounded once at the end.  ``own`` true: the
library's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64  # of the plain form

# The ranges the drawn cases are taken from: the largest listed sequence work in token-heads.
MOST_FWD, MOST_BWD, MOST_NORM = 1 << 20, 1 << 19, 1 << 26


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # prefill of continued prompts in fp32 (states in and out), the 2 x 4 x 2048 shape
        dict(name="delta_fwd_fp32_d64", op="fwd", dtype="f32", B=2, H=4, Hk=4, T=2048, dk=64, dv=64,
             gate=3.0, gate_sd=1.0, packed=False, states=True),
        # a packed training batch of odd length, two value heads to a key head: documents begin
        # with a closed gate, and the padding at the end has beta 0
        dict(name="delta_fwd_packed_bf16_d128", op="fwd", dtype="bf16", B=3, H=8, Hk=4, T=1111, dk=128, dv=128,
             gate=4.0, gate_sd=1.0, packed=True, states=False),
        # a training batch
        dict(name="delta_fwd_bf16_d128", op="fwd", dtype="bf16", B=8, H=16, Hk=16, T=4096, dk=128, dv=128,
             gate=4.0, gate_sd=1.0, packed=False, states=False),
        # one long sequence: few units, many chunks
        dict(name="delta_fwd_long_bf16_d128", op="fwd", dtype="bf16", B=1, H=16, Hk=16, T=65536, dk=128, dv=128,
             gate=5.0, gate_sd=1.5, packed=False, states=False),
        # gradients of a small packed fp32 model with shared key heads, odd length
        dict(name="delta_bwd_packed_fp32_d32", op="bwd", dtype="f32", B=2, H=6, Hk=2, T=777, dk=32, dv=32,
             gate=3.0, gate_sd=1.0, packed=True, states=False),
        # gradients of the training batch
        dict(name="delta_bwd_bf16_d128", op="bwd", dtype="bf16", B=8, H=16, Hk=16, T=4096, dk=128, dv=128,
             gate=4.0, gate_sd=1.0, packed=False, states=False),
        # one user's next token: latency
        dict(name="delta_step_1_bf16_d128", op="step", dtype="bf16", N=1, H=16, Hk=16, dk=128, dv=128,
             gate=4.0, gate_sd=1.0),
        # a serving batch's next tokens: the states' traffic
        dict(name="delta_step_256_bf16_d128", op="step", dtype="bf16", N=256, H=16, Hk=16, dk=128, dv=128,
             gate=4.0, gate_sd=1.0),
        # the block boundary of a small decoding batch (16 heads of 128 channels)
        dict(name="norm_fwd_rows8_bf16", op="norm_fwd", dtype="bf16", N=8, D=2048, post=True, gated=True, scaled=True,
             residual=True, pre=True),
        # the block boundary of the training batch
        dict(name="norm_fwd_bf16_d2048", op="norm_fwd", dtype="bf16", N=32768, D=2048, post=True, gated=True,
             scaled=True, residual=True, pre=True),
        # gradients of a gated per-head output norm, fp32 heads of 64 channels: short rows
        dict(name="norm_bwd_heads_fp32_d64", op="norm_bwd", dtype="f32", N=16384, D=64, post=True, gated=True,
             scaled=False, residual=False, pre=False),
        # gradients of the training batch's block boundary
        dict(name="norm_bwd_bf16_d2048", op="norm_bwd", dtype="bf16", N=32768, D=2048, post=True, gated=True,
             scaled=True, residual=True, pre=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    Hk = _log_int(rng, 1, 16)
    return Hk * rng.choice([1, 1, 1, 2, 4]), Hk


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    gate = dict(gate=round(rng.uniform(2.0, 6.0), 2), gate_sd=round(rng.uniform(0.5, 1.5), 2))
    if op in ("fwd", "bwd"):
        d = rng.choice([128, 128, 64]) if dtype == "bf16" else rng.choice([16, 32, 64, 128])
        H, Hk = _heads(rng)
        B = _log_int(rng, 1, 8)
        most = (MOST_FWD if op == "fwd" else MOST_BWD) // (B * H)
        if d < 128 or dtype == "f32":
            most //= 8
        T = _log_int(rng, 1 if op == "fwd" else 8, max(16, min(65536, most)))
        return dict(op=op, dtype=dtype, B=B, H=H, Hk=Hk, T=T, dk=d, dv=d, packed=rng.random() < 0.4,
                    states=dtype == "f32" and op == "fwd" and rng.random() < 0.5, **gate)
    if op == "step":
        d = rng.choice([128, 128, 64, 32])
        H, Hk = _heads(rng)
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, 4096 // H), H=H, Hk=Hk, dk=d, dv=d, **gate)
    D = rng.choice([64, 128, 1000, 2048, 2048, _log_int(rng, 33, 8192)])
    N = _log_int(rng, 1, min(524288, MOST_NORM // D))
    residual = rng.random() < 0.7
    return dict(op=op, dtype=dtype, N=N, D=D, post=not residual or rng.random() < 0.8, gated=rng.random() < 0.7,
                scaled=rng.random() < 0.6, residual=residual, pre=residual and rng.random() < 0.8)


# ---- inputs -----------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _delta_inputs(case, g, heads, shared):
    """q, k (unit rows of leading shape `shared`), v, gamma and beta (leading shape `heads`)."""
    dt, dk, dv = _dtype(case), case["dk"], case["dv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-12)

    s = dict(q=unit(normal(*shared, dk)).to(dt), k=unit(normal(*shared, dk)).to(dt), v=normal(*heads, dv).to(dt),
             gamma=torch.sigmoid(case["gate"] + case["gate_sd"] * normal(*heads)),
             beta=torch.sigmoid(normal(*heads)), scale=dk ** -0.5)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op, dt = case["op"], _dtype(case)
    if op in ("fwd", "bwd"):
        B, H, Hk, T, dk, dv = (case[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
        s = _delta_inputs(case, g, (B, H, T), (B, Hk, T))
        if case["packed"]:  # documents of a few hundred tokens; up to an eighth is padding
            first = torch.rand((B, 1, T), generator=g, device="cuda") < 1.0 / 200
            s["gamma"] = torch.where(first, 0.0, s["gamma"]).contiguous()
            used = T - (torch.rand((B, 1, 1), generator=g, device="cuda") * (T / 8)).long()
            pad = torch.arange(T, device="cuda") >= used
            s["beta"] = torch.where(pad, 0.0, s["beta"]).contiguous()
        s["S0"] = None
        s["S_final"] = None
        if case["states"]:
            s["S0"] = 0.3 * torch.randn((B, H, dv, dk), generator=g, device="cuda")
            s["S_final"] = torch.empty((B, H, dv, dk), device="cuda")
        if op == "bwd":
            s["dout"] = torch.randn((B, H, T, dv), generator=g, device="cuda").to(dt)
    elif op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        s = _delta_inputs(case, g, (N, H), (N, Hk))
        s["S"] = 0.3 * torch.randn((N, H, dv, dk), generator=g, device="cuda")
    else:
        N, D = case["N"], case["D"]

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        s = dict(x=(2.0 * normal(N, D)).to(dt) if case["residual"] else None, y=normal(N, D).to(dt),
                 gate=normal(N, D).to(dt) if case["gated"] else None,
                 w_post=1.0 + 0.1 * normal(D) if case["post"] else None,
                 res_scale=0.5 + 0.1 * normal(D) if case["scaled"] else None,
                 w_pre=1.0 + 0.1 * normal(D) if case["pre"] else None)
        if op == "norm_bwd":
            s["dx_out"] = normal(N, D).to(dt)
            s["dh"] = normal(N, D).to(dt) if case["pre"] else None
    s["op"] = op
    if own:
        from mesa_layer_gb300 import binding
        s["lib"] = binding
        if op in ("fwd", "bwd"):  # the workspace that a training or serving loop keeps
            size = binding.mesa_delta_workspace_size if op == "fwd" else binding.mesa_delta_backward_workspace_size
            n = size(case["B"], case["H"], case["Hk"], case["T"], case["dk"], case["dv"], s["q"].dtype)
            s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        elif op == "norm_bwd":
            n = binding.mesa_block_norm_backward_workspace_size(case["N"], case["D"])
            s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# ---- the plain forms (fp32, rounded once) -------------------------------------------------------
def _chunks(s):
    """fp32 inputs in chunks [U, NC, C, .] (the tail padded with tokens that do nothing) and what
    a chunk's algebra needs of them: the decays between its tokens, the strictly lower products
    k_i . k_j and the inverse of the unit lower triangular matrix I + diag(beta) (K K^T o D)."""
    B, H, T = s["gamma"].shape
    U, C = B * H, CHUNK
    NC = -(-T // C)
    group = H // s["q"].shape[1]

    def rows(x, shared=False):
        x = x.float()
        if shared and group > 1:
            x = x.repeat_interleave(group, dim=1)
        x = x.reshape(U, T, x.shape[-1])
        return torch.nn.functional.pad(x, (0, 0, 0, NC * C - T)).view(U, NC, C, x.shape[-1])

    def gates(x, fill):
        return torch.nn.functional.pad(x.float().reshape(U, T), (0, NC * C - T), value=fill).view(U, NC, C)

    c = dict(q=rows(s["q"], True), k=rows(s["k"], True), v=rows(s["v"]), beta=gates(s["beta"], 0.0),
             gamma=gates(s["gamma"], 1.0), U=U, NC=NC, T=T, group=group)
    # log-decays from the chunk's start; closed gates are counted apart, so that a zero gate
    # cuts exactly
    shut = c["gamma"] <= 0
    lg = torch.log(torch.where(shut, 1.0, c["gamma"])).cumsum(-1)
    z = shut.cumsum(-1)
    low = torch.ones(C, C, device=lg.device).tril().bool()

    def decay(l_i, z_i, l_j, z_j, mask):
        keep = mask & (z_i == z_j)
        return torch.exp(torch.where(keep, l_i - l_j, -math.inf))

    c["D"] = decay(lg[..., :, None], z[..., :, None], lg[..., None, :], z[..., None, :], low)  # j <= i
    c["from0"] = torch.where(z == 0, torch.exp(lg), 0.0)                     # chunk start -> i
    c["toC"] = torch.where(z == z[..., -1:], torch.exp(lg[..., -1:] - lg), 0.0)  # i -> chunk end
    c["all"] = c["from0"][..., -1]
    lp, zp = torch.nn.functional.pad(lg, (1, -1)), torch.nn.functional.pad(z, (1, -1))
    c["Dprev"] = decay(lp[..., :, None], zp[..., :, None], lg[..., None, :], z[..., None, :], low.tril(-1))
    c["from0prev"] = torch.where(zp == 0, torch.exp(lp), 0.0)
    c["KK"] = c["k"] @ c["k"].mT
    c["L"] = c["KK"] * c["D"].tril(-1)
    A = c["beta"][..., None] * c["L"]
    X = torch.eye(C, device=A.device).expand_as(A)
    i = torch.arange(C, device=A.device)
    size = 1
    while size < C:  # inverses of the diagonal blocks, doubled
        corner = ((i[:, None] // size) == (i[None, :] // size) + 1) & ((i[:, None] // size) % 2 == 1)
        X = X - X @ (A * corner) @ X
        size *= 2
    c["X"] = X
    return c


def _plain_chain(c, S, scale, keep=False):
    """The chunk recurrence: outputs, final state; with keep the states before each chunk and e."""
    qd, kd = scale * c["from0"][..., None] * c["q"], c["from0"][..., None] * c["k"]
    P = scale * (c["q"] @ c["k"].mT) * c["D"]
    Xb, kC = c["X"] * c["beta"][..., None, :], c["toC"][..., None] * c["k"]
    out, states, us = [], [], []
    for n in range(c["NC"]):
        if keep:
            states.append(S)
        u = Xb[:, n] @ (c["v"][:, n] - kd[:, n] @ S.mT)
        if keep:
            us.append(u)
        else:
            out.append(qd[:, n] @ S.mT + P[:, n] @ u)
        S = c["all"][:, n, None, None] * S + u.mT @ kC[:, n]
    if keep:
        return torch.stack(states, 1), torch.stack(us, 1), P, qd, kd, kC, Xb
    return torch.stack(out, 1), S


def _plain_fwd(s):
    B, H, T = s["gamma"].shape
    dt, dv, dk = s["q"].dtype, s["v"].shape[-1], s["q"].shape[-1]
    c = _chunks(s)
    S = s["S0"].reshape(B * H, dv, dk) if s["S0"] is not None else s["gamma"].new_zeros((B * H, dv, dk))
    out, S = _plain_chain(c, S, s["scale"])
    out = out.reshape(B, H, -1, dv)[:, :, :T].to(dt)
    if s["S_final"] is None:
        return {"out": out}
    s["S_final"].copy_(S.view(B, H, dv, dk))
    return {"out": out, "S_final": s["S_final"]}


def _plain_bwd(s):
    B, H, T = s["gamma"].shape
    dt, dv, dk, scale = s["q"].dtype, s["v"].shape[-1], s["q"].shape[-1], s["scale"]
    c = _chunks(s)
    U, NC = c["U"], c["NC"]
    g = torch.nn.functional.pad(s["dout"].float().reshape(U, T, dv), (0, 0, 0, NC * CHUNK - T)).view(U, NC, CHUNK, dv)
    S0, u, P, qd, kd, kC, Xb = _plain_chain(c, s["gamma"].new_zeros((U, dv, dk)), scale, keep=True)
    e = c["v"] - kd @ S0.mT - c["L"] @ u
    # the adjoint chain: du_t, and the adjoint of the state after each chunk
    Pg, qg, Xt, kb = P.mT @ g, g.mT @ qd, c["X"].mT, kd * c["beta"][..., None]
    dS, dSs, dus = s["gamma"].new_zeros((U, dv, dk)), [None] * NC, [None] * NC
    for n in range(NC - 1, -1, -1):
        dSs[n] = dS
        dus[n] = Xt[:, n] @ (Pg[:, n] + kC[:, n] @ dS.mT)
        dS = c["all"][:, n, None, None] * dS + qg[:, n] - dus[n].mT @ kb[:, n]
    dS, du = torch.stack(dSs, 1), torch.stack(dus, 1)
    db = du * c["beta"][..., None]
    gu, bu = scale * (g @ u.mT), db @ u.mT
    W, V = gu * c["D"], bu * c["D"].tril(-1)
    gS, bS, uS = scale * (g @ S0), db @ S0, u @ dS
    dq = c["from0"][..., None] * gS + W @ c["k"]
    dk_ = W.mT @ c["q"] + c["toC"][..., None] * uS - c["from0"][..., None] * bS - (V + V.mT) @ c["k"]
    dbeta = (du * e).sum(-1)
    # dgamma_t: every product that crosses the gate t, without its own decay
    x_in = (gS * c["q"]).sum(-1) - (bS * c["k"]).sum(-1)           # i against the state before the chunk
    x_out = (uS * c["k"]).sum(-1)                                   # j against the adjoint after it
    X = gu * (c["q"] @ c["k"].mT) - bu * c["KK"]
    Dm = c["D"].mT                                                  # [t, i]: decay t -> i, i >= t
    dgamma = c["from0prev"] * (Dm @ x_in[..., None])[..., 0] + ((Dm @ X) * c["Dprev"]).sum(-1)
    dgamma += c["toC"] * (c["from0prev"] * (dS * S0).sum((-1, -2))[..., None] + (c["Dprev"] @ x_out[..., None])[..., 0])

    def back(x, shared=False):
        x = x.reshape(B, H, NC * CHUNK, -1)[:, :, :T]
        if shared and c["group"] > 1:
            x = x.view(B, -1, c["group"], T, x.shape[-1]).sum(2)
        return x.to(dt)

    return {"dq": back(dq, True), "dk": back(dk_, True), "dv": back(db), "dgamma": back(dgamma)[..., 0],
            "dbeta": back(dbeta)[..., 0]}


def _plain_step(s):
    S, dt = s["S"], s["q"].dtype
    group = S.shape[1] // s["q"].shape[1]
    q, k = (x.float().repeat_interleave(group, dim=1) for x in (s["q"], s["k"]))
    S.mul_(s["gamma"][..., None, None])
    u = s["beta"][..., None] * (s["v"].float() - (S @ k[..., None])[..., 0])
    S.add_(u[..., :, None] * k[..., None, :])
    return {"out": (s["scale"] * (S @ q[..., None])[..., 0]).to(dt), "S": S}


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _norm_parts(s):
    y = s["y"].float()
    D = y.shape[-1]
    r_post = torch.rsqrt(y.square().sum(-1, keepdim=True) / D + EPS) if s["w_post"] is not None else None
    yn = y * r_post if r_post is not None else y
    z = yn * s["w_post"] if r_post is not None else y
    a = _silu(s["gate"].float()) if s["gate"] is not None else None
    t = z if a is None else a * z
    X = t if s["res_scale"] is None else s["res_scale"] * t
    if s["x"] is not None:
        X = s["x"].float() + X
    r_pre = torch.rsqrt(X.square().sum(-1, keepdim=True) / D + EPS) if s["w_pre"] is not None else None
    return D, r_post, yn, z, a, t, X, r_pre


def _plain_norm_fwd(s):
    _, _, _, _, _, _, X, r_pre = _norm_parts(s)
    dt = s["y"].dtype
    r = {"x_out": X.to(dt)}
    if r_pre is not None:
        r["h"] = (X * r_pre * s["w_pre"]).to(dt)
    return r


def _plain_norm_bwd(s):
    D, r_post, yn, z, a, t, X, r_pre = _norm_parts(s)
    dt = s["y"].dtype
    dX = s["dx_out"].float()
    r = {}
    if r_pre is not None:
        Xn, dh = X * r_pre, s["dh"].float()
        r["dw_pre"] = (dh * Xn).sum(0)
        d = dh * s["w_pre"]
        dX = dX + r_pre * (d - Xn * ((d * Xn).sum(-1, keepdim=True) / D))
    if s["x"] is not None:
        r["dx"] = dX.to(dt)
    if s["res_scale"] is not None:
        r["dres_scale"] = (dX * t).sum(0)
        dX = dX * s["res_scale"]
    if a is not None:
        gate = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        r["dgate"] = (dX * z * sig * (1.0 + gate * (1.0 - sig))).to(dt)
        dX = dX * a
    if r_post is not None:
        r["dw_post"] = (dX * yn).sum(0)
        d = dX * s["w_post"]
        dX = r_post * (d - yn * ((d * yn).sum(-1, keepdim=True) / D))
    r["dy"] = dX.to(dt)
    return r


# ---- the library's calls ------------------------------------------------------------------------
def _own(s):
    lib, op = s["lib"], s["op"]
    if op == "fwd":
        out = lib.mesa_delta_forward_chunked(s["q"], s["k"], s["v"], s["gamma"], s["beta"], scale=s["scale"],
                                             S0=s["S0"], S_final=s["S_final"], workspace=s["workspace"])
        return {"out": out} if s["S_final"] is None else {"out": out, "S_final": s["S_final"]}
    if op == "bwd":
        return dict(zip(("dq", "dk", "dv", "dgamma", "dbeta"), lib.mesa_delta_backward_chunked(
            s["q"], s["k"], s["v"], s["gamma"], s["beta"], s["dout"], scale=s["scale"], workspace=s["workspace"])))
    if op == "step":
        return {"out": lib.mesa_delta_step(s["S"], s["q"], s["k"], s["v"], s["gamma"], s["beta"], scale=s["scale"]),
                "S": s["S"]}
    if op == "norm_fwd":
        r = lib.mesa_block_norm(s["x"], s["y"], gate=s["gate"], w_post=s["w_post"], res_scale=s["res_scale"],
                                w_pre=s["w_pre"], eps=EPS)
        return {k: v for k, v in zip(("x_out", "h"), r) if v is not None}
    r = lib.mesa_block_norm_backward(s["x"], s["y"], s["dx_out"], dh=s["dh"], gate=s["gate"], w_post=s["w_post"],
                                     res_scale=s["res_scale"], w_pre=s["w_pre"], eps=EPS, workspace=s["workspace"])
    return {k: v for k, v in zip(("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre"), r) if v is not None}


PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd,
         "norm_bwd": _plain_norm_bwd}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------------------
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("fwd", "bwd"):
        B, H, Hk, T, dk, dv = (case[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
        qk, vo, gates = B * Hk * T * dk * esz, B * H * T * dv * esz, 4 * B * H * T
        if op == "fwd":  # q, k, v, gates in, o out; S k, u k^T and S q of each token
            return {"bytes": 2 * qk + 2 * vo + 2 * gates + (8 * B * H * dk * dv if case["states"] else 0),
                    "flops": 6.0 * B * H * T * dk * dv}
        # q, k, v, dout, gates in, their gradients out; the states again (4), the adjoints
        # dS k, du k^T, dO q^T (6), dq and dk from them (6), dgamma (2)
        return {"bytes": 4 * qk + 3 * vo + 2 * gates + 2 * B * H * T * esz, "flops": 18.0 * B * H * T * dk * dv}
    if op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        return {"bytes": 8 * N * H * dk * dv + esz * (2 * N * Hk * dk + 2 * N * H * dv) + 8 * N * H,
                "flops": 6.0 * N * H * dk * dv}
    n = case["N"] * case["D"]
    reads = 1 + case["residual"] + case["gated"]
    if op == "norm_fwd":
        return {"bytes": n * esz * (reads + 1 + case["pre"]) + 4 * case["D"] * (case["post"] + case["scaled"] + case["pre"]),
                "flops": 12.0 * n}
    writes = reads
    return {"bytes": n * esz * (reads + 1 + case["pre"] + writes) + 8 * case["D"] * (case["post"] + case["scaled"] + case["pre"]),
            "flops": 30.0 * n}


# ---- the definitions in 64 bits -------------------------------------------------------------------
def _exact_inputs(s):
    """Token-major fp64 views [T, U, .] of a sequence case."""
    B, H, T = s["gamma"].shape
    group = H // s["q"].shape[1]

    def seq(x, shared=False):
        x = x.double()
        if shared:
            x = x.repeat_interleave(group, dim=1)
        return x.reshape(B * H, T, -1).transpose(0, 1).contiguous()

    return (seq(s["q"], True), seq(s["k"], True), seq(s["v"]), seq(s["gamma"][..., None]), seq(s["beta"][..., None]),
            B, H, T, group)


def _exact_seq(s, op):
    q, k, v, gamma, beta, B, H, T, group = _exact_inputs(s)
    U, dv, dk, scale = B * H, v.shape[-1], k.shape[-1], s["scale"]
    S = s["S0"].double().reshape(U, dv, dk).clone() if s["S0"] is not None else v.new_zeros((U, dv, dk))

    def step(S, t):
        """S_t in place of S_{t-1}; e_t."""
        S.mul_(gamma[t][..., None])
        e = torch.baddbmm(v[t][..., None], S, k[t][..., None], alpha=-1.0)[..., 0]
        S.baddbmm_((beta[t] * e)[..., None], k[t][:, None, :])
        return e

    if op == "fwd":
        out = torch.empty_like(v)
        for t in range(T):
            step(S, t)
            torch.mul(torch.bmm(S, q[t][..., None])[..., 0], scale, out=out[t])
        r = {"out": out.transpose(0, 1).reshape(B, H, T, dv)}
        if s["S_final"] is not None:
            r["S_final"] = S.view(B, H, dv, dk)
        return r
    span = 32
    saved = []
    for t in range(T):
        if t % span == 0:
            saved.append(S.clone())
        step(S, t)
    g = s["dout"].double().reshape(U, T, dv).transpose(0, 1).contiguous()
    dq, dk_, dv_, dgam, dbet = (torch.empty_like(x) for x in (q, k, v, gamma, beta))
    A = torch.zeros_like(S)  # adjoint of S_t from the tokens after t
    for first in range((T - 1) // span * span, -1, -span):
        last = min(T, first + span)
        states, es = [saved[first // span]], []
        for t in range(first, last):
            S = states[-1].clone()
            es.append(step(S, t))
            states.append(S)
        for t in range(last - 1, first - 1, -1):
            before, after, e = states[t - first], states[t - first + 1], es[t - first]
            dq[t] = scale * (after.mT @ g[t][..., None])[..., 0]
            A.baddbmm_(g[t][..., None], q[t][:, None, :], alpha=scale)
            du = (A @ k[t][..., None])[..., 0]
            dbet[t] = (du * e).sum(-1, keepdim=True)
            dv_[t] = beta[t] * du
            dk_[t] = (A.mT @ (beta[t] * e)[..., None])[..., 0] - gamma[t] * (before.mT @ dv_[t][..., None])[..., 0]
            A.baddbmm_(dv_[t][..., None], k[t][:, None, :], alpha=-1.0)
            dgam[t] = (A * before).sum((-1, -2))[:, None]
            A.mul_(gamma[t][..., None])

    def back(x, shared=False):
        x = x.transpose(0, 1).reshape(B, H, T, -1)
        return x.view(B, H // group, group, T, x.shape[-1]).sum(2) if shared else x

    return {"dq": back(dq, True), "dk": back(dk_, True), "dv": back(dv_), "dgamma": back(dgam)[..., 0],
            "dbeta": back(dbet)[..., 0]}


def _exact_norm(s, op):
    t = {k: s[k].double().requires_grad_(op == "norm_bwd") for k in ("x", "y", "gate", "w_post", "res_scale", "w_pre")
         if s[k] is not None}
    X = t["y"]
    if "w_post" in t:
        X = X / (X.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * t["w_post"]
    if "gate" in t:
        X = X * t["gate"] * torch.sigmoid(t["gate"])
    if "res_scale" in t:
        X = X * t["res_scale"]
    if "x" in t:
        X = X + t["x"]
    h = X / (X.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * t["w_pre"] if "w_pre" in t else None
    if op == "norm_fwd":
        return {"x_out": X} if h is None else {"x_out": X, "h": h}
    L = (X * s["dx_out"].double()).sum()
    if h is not None:
        L = L + (h * s["dh"].double()).sum()
    return {"d" + k: x for k, x in zip(t, torch.autograd.grad(L, list(t.values())))}


def exact(case, seed):
    op = case["op"]
    if op == "bwd" and case["T"] > 32768:  # a token at a time: too long
        return None
    s = prepare(case, seed)
    if op in ("fwd", "bwd"):
        return _exact_seq(s, op)
    if op == "step":
        group = case["H"] // case["Hk"]
        q, k = (x.double().repeat_interleave(group, dim=1) for x in (s["q"], s["k"]))
        S = s["S"].double() * s["gamma"].double()[..., None, None]
        e = s["v"].double() - torch.einsum("nhvk,nhk->nhv", S, k)
        S = S + torch.einsum("nh,nhv,nhk->nhvk", s["beta"].double(), e, k)
        return {"out": s["scale"] * torch.einsum("nhvk,nhk->nhv", S, q), "S": S}
    return _exact_norm(s, op)
