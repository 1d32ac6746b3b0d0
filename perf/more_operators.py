"""Cases of the selective state space scan (chunked forward, backward, decode step), of the short causal convolution
in front of it (forward, backward, decode step) and of the per-head norm with position rotation of queries and keys
(forward, backward), and their plain forms.

Scan, per (batch, head) unit, state S [dv, dk], zero (or given) before token 0; q, k and v are what the scan's
literature calls C, B and x:
    D_t = softplus(dt_t + dt_bias_h),   a_t = exp(D_t A_h)  (0 where a document starts),
    S_t = a_t S_{t-1} + D_t v_t k_t^T,  o_t = S_t q_t + skip_h v_t.
q and k may have fewer heads than v (Hk divides H; head h reads head h // (H / Hk)).

Convolution, per (batch, head) unit and channel, W taps; inputs before the first token of a document are zero (before
the sequence: zero or given):
    y_t = bias + sum_s w_s x_{t-s},     o_t = y_t or silu(y_t).

Norm and rotation, per row x of d channels: n = x rsqrt(mean(x^2) + eps) w; the first R channels of n turn by the
angles pos f_j in pairs (j, j + R/2) or (2j, 2j + 1), scaled by rot_scale.

``own`` false: elementary torch operations in fp32 (log-decays and angles in fp64), rounded once at the end.  ``own``
true: the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64  # of the plain scan

# The ranges the drawn cases are taken from: the largest listed sequence work in token-heads, and elements.
MOST_FWD, MOST_BWD, MOST_CONV = 1 << 20, 1 << 19, 1 << 26


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # prefill of continued prompts in fp32 (states in and out), the 2 x 4 x 2048 shape
        dict(name="ssm_fwd_fp32_d64", op="fwd", dtype="f32", B=2, H=4, Hk=4, T=2048, dk=64, dv=64, packed=False,
             states=True, skip=True),
        # a packed training batch of odd length, four value heads of 64 channels to a key head; padding at the end
        dict(name="ssm_fwd_packed_bf16", op="fwd", dtype="bf16", B=3, H=8, Hk=2, T=1111, dk=128, dv=64, packed=True,
             states=False, skip=True),
        # a training batch
        dict(name="ssm_fwd_bf16_d128", op="fwd", dtype="bf16", B=8, H=16, Hk=16, T=4096, dk=128, dv=128, packed=False,
             states=False, skip=True),
        # one long prompt whose state goes on to decoding: few units, many chunks
        dict(name="ssm_fwd_long_bf16_d128", op="fwd", dtype="bf16", B=1, H=16, Hk=16, T=65536, dk=128, dv=128,
             packed=False, states=True, skip=True),
        # gradients of a small packed fp32 model with shared key heads, odd length
        dict(name="ssm_bwd_packed_fp32_d32", op="bwd", dtype="f32", B=2, H=6, Hk=2, T=777, dk=32, dv=32, packed=True,
             states=False, skip=True),
        # gradients of the training batch
        dict(name="ssm_bwd_bf16_d128", op="bwd", dtype="bf16", B=8, H=16, Hk=16, T=4096, dk=128, dv=128, packed=False,
             states=False, skip=True),
        # one user's next token: latency
        dict(name="ssm_step_1_bf16_d128", op="step", dtype="bf16", N=1, H=16, Hk=16, dk=128, dv=128, skip=True),
        # a serving batch's next tokens: the states' traffic
        dict(name="ssm_step_256_bf16_d128", op="step", dtype="bf16", N=256, H=16, Hk=16, dk=128, dv=128, skip=True),
        # the convolution of the training batch's channels
        dict(name="conv_fwd_bf16", op="conv", dtype="bf16", B=8, H=16, T=4096, d=128, W=4, silu=True, packed=False),
        # its gradients, for packed documents of odd length
        dict(name="conv_bwd_packed_bf16", op="conv_bwd", dtype="bf16", B=8, H=16, T=4001, d=128, W=4, silu=True,
             packed=True),
        # queries and keys of a serving batch's next tokens, each at its own position of a long context
        dict(name="rotary_step_bf16_d128", op="rot", dtype="bf16", B=256, H=16, Hk=4, T=1, d=128, R=128, interleaved=False,
             norm=True, far=1 << 20),
        # gradients of the training batch's queries and keys, half of the channels rotated
        dict(name="rotary_bwd_bf16_d128", op="rot_bwd", dtype="bf16", B=8, H=16, Hk=16, T=4096, d=128, R=64,
             interleaved=True, norm=True, far=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    Hk = _log_int(rng, 1, 16)
    group = rng.choice([1, 1, 1, 2, 4])
    return Hk * max(group, -(-4 // Hk)), Hk  # four heads at least


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "step", "conv", "conv_bwd", "conv_step", "rot", "rot_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("fwd", "bwd"):
        if dtype == "bf16":
            dk, dv = rng.choice([(128, 128), (128, 64), (128, 128), (64, 64)])
        else:
            dk, dv = rng.choice([(16, 16), (32, 32), (64, 64), (128, 128), (128, 64), (16, 64)])
        H, Hk = _heads(rng)
        B = _log_int(rng, 1, 8)
        most = (MOST_FWD if op == "fwd" else MOST_BWD) // (B * H)
        if dk < 128 or dtype == "f32":
            most //= 8
        return dict(op=op, dtype=dtype, B=B, H=H, Hk=Hk, T=_log_int(rng, 1, max(16, min(65536, most))), dk=dk, dv=dv,
                    packed=rng.random() < 0.4, states=op == "fwd" and rng.random() < 0.5, skip=rng.random() < 0.7)
    if op == "step":
        d = rng.choice([128, 128, 64, 32])
        H, Hk = _heads(rng)
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, 4096 // H), H=H, Hk=Hk, dk=d, dv=rng.choice([d, 64]),
                    skip=rng.random() < 0.7)
    if op in ("conv", "conv_bwd", "conv_step"):
        H = rng.choice([1, 4, 16, _log_int(rng, 1, 32)])
        d = rng.choice([64, 128, 128, 8 * _log_int(rng, 1, 64)])
        B = _log_int(rng, 1, 256 if op == "conv_step" else 8)
        T = 1 if op == "conv_step" else _log_int(rng, 1, max(2, min(65536, MOST_CONV // (B * H * d))))
        return dict(op=op, dtype=dtype, B=B, H=H, T=T, d=d, W=rng.choice([2, 3, 4, 4, 8]), silu=rng.random() < 0.8,
                    packed=op != "conv_step" and rng.random() < 0.4)
    H, Hk = _heads(rng)
    d = rng.choice([64, 128, 128, 32])
    B = _log_int(rng, 1, 64)
    T = _log_int(rng, 1, max(2, min(65536, MOST_CONV // (B * (H + Hk) * d))))
    return dict(op=op, dtype=dtype, B=B, H=H, Hk=Hk, T=T, d=d, R=rng.choice([d, d, d // 2, d // 4]),
                interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, far=rng.choice([0, 0, 1 << 20]))


# ---- inputs -----------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _starts(case, g):
    """Documents of a few hundred tokens."""
    return torch.rand((case["B"], case["T"]), generator=g, device="cuda") < 1.0 / 200 if case["packed"] else None


def _scan_inputs(case, g, heads, shared):
    dt, H, dk, dv = _dtype(case), case["H"], case["dk"], case["dv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand((H,), generator=g, device="cuda")

    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1)))  # a head's usual step
    return dict(q=(dk ** -0.5 * normal(*shared, dk)).to(dt), k=normal(*shared, dk).to(dt), v=normal(*heads, dv).to(dt),
                dt=0.7 * normal(*heads), A=-uniform(1.0, 16.0), dt_bias=step + torch.log(-torch.expm1(-step)),
                skip=1.0 + 0.1 * normal(H) if case["skip"] else None)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    op, dt = case["op"], _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op in ("fwd", "bwd"):
        B, H, Hk, T, dk, dv = (case[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
        s = _scan_inputs(case, g, (B, H, T), (B, Hk, T))
        s["starts"] = _starts(case, g)
        if case["packed"]:  # up to an eighth is padding: steps of zero length
            used = T - (torch.rand((B, 1, 1), generator=g, device="cuda") * (T / 8)).long()
            s["dt"] = torch.where(torch.arange(T, device="cuda") >= used, -math.inf, s["dt"]).contiguous()
        s["S0"] = 0.3 * normal(B, H, dv, dk) if case["states"] else None
        s["S_final"] = torch.empty((B, H, dv, dk), device="cuda") if case["states"] else None
        if op == "bwd":
            s["dout"] = normal(B, H, T, dv).to(dt)
    elif op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        s = _scan_inputs(case, g, (N, H), (N, Hk))
        s["S"] = 0.3 * normal(N, H, dv, dk)
    elif op in ("conv", "conv_bwd", "conv_step"):
        B, H, T, d, W = (case[n] for n in ("B", "H", "T", "d", "W"))
        s = dict(x=normal(B, H, T, d).to(dt), w=W ** -0.5 * normal(H, d, W), bias=0.2 * normal(H, d), silu=case["silu"])
        s["starts"] = _starts(case, g)
        if op == "conv_bwd":
            s["dout"] = normal(B, H, T, d).to(dt)
        if op == "conv_step":
            s["x"] = s["x"][:, :, 0].contiguous()
            s["state"] = normal(B, H, W - 1, d)
    else:
        B, H, Hk, T, d, R = (case[n] for n in ("B", "H", "Hk", "T", "d", "R"))
        s = dict(q=normal(B, H, T, d).to(dt), k=normal(B, Hk, T, d).to(dt), interleaved=case["interleaved"],
                 norm=case["norm"], rot_scale=1.0, wq=None, wk=None, positions=None,
                 inv_freq=torch.tensor([10000.0 ** (-2.0 * j / R) for j in range(R // 2)], device="cuda"))
        if case["norm"]:
            s["wq"], s["wk"] = 1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)
        if case["far"]:  # sequences that begin anywhere in a long context, frequencies scaled for it
            first = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
            s["inv_freq"], s["rot_scale"] = s["inv_freq"] / 8.0, 1.2
        if op == "rot_bwd":
            s["dq_out"], s["dk_out"] = normal(B, H, T, d).to(dt), normal(B, Hk, T, d).to(dt)
    s["op"] = op
    if own:
        from mesa_layer_gb300 import binding
        s["lib"] = binding
        size = None  # the workspace that a training or serving loop keeps
        if op in ("fwd", "bwd"):
            size = (binding.mesa_ssm_workspace_size if op == "fwd" else binding.mesa_ssm_backward_workspace_size)(
                case["B"], case["H"], case["Hk"], case["T"], case["dk"], case["dv"], s["q"].dtype)
        elif op == "conv_bwd":
            size = binding.mesa_causal_conv_backward_workspace_size(case["B"], case["H"], case["T"], case["d"], case["W"])
        elif op == "rot_bwd":
            size = binding.mesa_qk_norm_rotary_backward_workspace_size(case["B"], case["H"], case["Hk"], case["T"], case["d"])
        if size is not None:
            s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


# ---- the plain forms (fp32, rounded once) -------------------------------------------------------
def _softplus(x):
    return x.clamp_min(0.0) + torch.log1p(torch.exp(-x.abs()))


def _chunks(s):
    """fp32 inputs in chunks [U, NC, C, .] (the tail padded with tokens that do nothing) and their decays: D[i, j] from
    token j to token i >= j, first[i] from before the chunk, last[j] to its end, E[m, n] from after n chunks to after m."""
    B, H, T = s["dt"].shape
    U, C, NC = B * H, CHUNK, -(-T // CHUNK)
    group = H // s["q"].shape[1]

    def rows(x, shared=False):
        x = x.float()
        if shared and group > 1:
            x = x.repeat_interleave(group, dim=1)
        return torch.nn.functional.pad(x.reshape(U, T, x.shape[-1]), (0, 0, 0, NC * C - T)).view(U, NC, C, x.shape[-1])

    def tokens(x):
        return torch.nn.functional.pad(x.expand(B, H, T).reshape(U, T), (0, NC * C - T)).view(U, NC, C)

    raw = s["dt"] + s["dt_bias"][:, None]
    step = _softplus(raw)
    la = tokens((step.double() * s["A"].double()[:, None])).view(U, -1).cumsum(-1).view(U, NC, C)
    z = tokens(s["starts"][:, None].long() if s["starts"] is not None else torch.zeros_like(s["dt"], dtype=torch.long))
    z = z.view(U, -1).cumsum(-1).view(U, NC, C)

    def decay(l_i, z_i, l_j, z_j, mask=None):
        keep = z_i == z_j if mask is None else mask & (z_i == z_j)
        return torch.exp(torch.where(keep, l_i - l_j, -math.inf).float())

    low = torch.ones(C, C, device=la.device).tril().bool()
    end_l = torch.nn.functional.pad(la[..., -1], (1, 0))  # after 0, 1, ... NC chunks
    end_z = torch.nn.functional.pad(z[..., -1], (1, 0))
    below = torch.ones(NC + 1, NC + 1, device=la.device).tril().bool()
    return dict(q=rows(s["q"], True), k=rows(s["k"], True), v=rows(s["v"]), step=tokens(step), U=U, NC=NC, group=group,
                low=low, raw=raw, D=decay(la[..., :, None], z[..., :, None], la[..., None, :], z[..., None, :], low),
                first=decay(la, z, end_l[:, :-1, None], end_z[:, :-1, None]),
                last=decay(end_l[:, 1:, None], end_z[:, 1:, None], la, z),
                E=decay(end_l[:, :, None], end_z[:, :, None], end_l[:, None, :], end_z[:, None, :], below))


def _states(c, s):
    """The states after 0, 1, ... NC chunks [U, NC + 1, dv, dk], and what each token writes."""
    u = c["step"][..., None] * c["v"]
    added = (c["last"][..., None] * u).mT @ c["k"]
    S0 = added.new_zeros(added[:, :1].shape) if s["S0"] is None else s["S0"].reshape(c["U"], 1, *added.shape[2:])
    added = torch.cat([S0, added], 1)
    return (c["E"] @ added.flatten(2)).view(added.shape), u


def _plain_fwd(s):
    B, H, T = s["dt"].shape
    dv = s["v"].shape[-1]
    c = _chunks(s)
    S, u = _states(c, s)
    out = c["first"][..., None] * (c["q"] @ S[:, :-1].mT) + ((c["q"] @ c["k"].mT) * c["D"]) @ u
    out = out.reshape(B, H, -1, dv)[:, :, :T]
    if s["skip"] is not None:
        out = out + s["skip"][:, None, None] * s["v"].float()
    out = out.to(s["q"].dtype)
    if s["S_final"] is None:
        return {"out": out}
    s["S_final"].copy_(S[:, -1].view(s["S_final"].shape))
    return {"out": out, "S_final": s["S_final"]}


def _plain_bwd(s):
    B, H, T = s["dt"].shape
    dt, dv = s["q"].dtype, s["v"].shape[-1]
    c = _chunks(s)
    S, u = _states(c, s)
    g = torch.nn.functional.pad(s["dout"].float().reshape(c["U"], T, dv), (0, 0, 0, c["NC"] * CHUNK - T)).view(c["v"].shape)
    # the adjoints of the states after 0, 1, ... NC chunks
    given = (c["first"][..., None] * g).mT @ c["q"]
    given = torch.cat([given, torch.zeros_like(given[:, :1])], 1)
    R = (c["E"].mT @ given.flatten(2)).view(S.shape)
    S0, R1 = S[:, :-1], R[:, 1:]
    M, gu = (c["q"] @ c["k"].mT) * c["D"], g @ u.mT
    W = gu * c["D"]
    gS, kR, uR = g @ S0, c["k"] @ R1.mT, u @ R1
    dq = c["first"][..., None] * gS + W @ c["k"]
    dk = W.mT @ c["q"] + c["last"][..., None] * uR
    du = M.mT @ g + c["last"][..., None] * kR
    # d log a_t: every product that crosses the decay of token t
    X = M * gu
    x_in, x_out = c["first"] * (gS * c["q"]).sum(-1), c["last"] * (uR * c["k"]).sum(-1)
    upper, strict = c["low"].mT.float(), c["low"].tril(-1).float()  # [t, i]: i >= t; [t, j]: j < t
    across = c["E"].diagonal(-1, 1, 2) * (R1 * S0).sum((-1, -2))
    da = ((upper @ X) * strict).sum(-1) + (upper @ x_in[..., None])[..., 0] + (strict @ x_out[..., None])[..., 0]
    da = da + across[..., None]
    if s["starts"] is not None:  # the decay of a document's first token is zero whatever its step
        da = torch.where(torch.nn.functional.pad(s["starts"][:, None].expand(B, H, T).reshape(c["U"], T),
                                                 (0, c["NC"] * CHUNK - T)).view(da.shape), 0.0, da)

    def back(x, shared=False):
        x = x.reshape(B, H, c["NC"] * CHUNK, -1)[:, :, :T]
        return x.view(B, -1, c["group"], T, x.shape[-1]).sum(2) if shared and c["group"] > 1 else x

    step, da, du = back(c["step"])[..., 0], back(da)[..., 0], back(du)
    dstep = (du * s["v"].float()).sum(-1) + s["A"][:, None] * da
    draw_ = dstep * torch.sigmoid(c["raw"])
    r = {"dq": back(dq, True), "dk": back(dk, True), "dv": step[..., None] * du, "ddt": draw_,
         "dA": (step * da).sum((0, 2)), "ddt_bias": draw_.sum((0, 2))}
    if s["skip"] is not None:
        gv = s["dout"].float() * s["v"].float()
        r["dv"] = r["dv"] + s["skip"][:, None, None] * s["dout"].float()
        r["dskip"] = gv.sum(-1).sum((0, 2))
    return {n: x.to(dt) for n, x in r.items()}


def _plain_step(s):
    S, dt = s["S"], s["q"].dtype
    group = S.shape[1] // s["q"].shape[1]
    q, k = (x.float().repeat_interleave(group, dim=1) for x in (s["q"], s["k"]))
    step = _softplus(s["dt"] + s["dt_bias"])
    S.mul_(torch.exp(step * s["A"])[..., None, None])
    S.add_((step[..., None] * s["v"].float())[..., :, None] * k[..., None, :])
    out = (S @ q[..., None])[..., 0]
    if s["skip"] is not None:
        out = out + s["skip"][:, None] * s["v"].float()
    return {"out": out.to(dt), "S": S}


def _shifted(x, s, starts):
    """x s tokens back, zero where that is before the token's document."""
    if s == 0:
        return x
    y = torch.nn.functional.pad(x, (0, 0, s, 0))[:, :, : x.shape[2]]
    if starts is None:
        return y
    z = starts.long().cumsum(-1)
    same = z == torch.nn.functional.pad(z, (s, 0), value=-1)[:, : z.shape[1]]
    return torch.where(same[:, None, :, None], y, 0.0)


def _conv_sum(s):
    x, W = s["x"].float(), s["w"].shape[-1]
    return sum(s["w"][:, None, :, i] * _shifted(x, i, s["starts"]) for i in range(W)) + s["bias"][:, None]


def _plain_conv(s):
    y = _conv_sum(s)
    return {"out": (y * torch.sigmoid(y) if s["silu"] else y).to(s["x"].dtype)}


def _plain_conv_bwd(s):
    x, W, T = s["x"].float(), s["w"].shape[-1], s["x"].shape[2]
    dy = s["dout"].float()
    if s["silu"]:
        y = _conv_sum(s)
        sig = torch.sigmoid(y)
        dy = dy * sig * (1.0 + y * (1.0 - sig))
    dw = torch.stack([(dy * _shifted(x, i, s["starts"])).sum(2).sum(0) for i in range(W)], -1)
    z = s["starts"].long().cumsum(-1) if s["starts"] is not None else torch.zeros_like(x[:, 0, :, 0], dtype=torch.long)

    def ahead(i):  # dy i tokens on, zero past the token's document
        same = z == torch.nn.functional.pad(z, (0, i), value=-1)[:, i:]
        return torch.where(same[:, None, :, None], torch.nn.functional.pad(dy, (0, 0, 0, i))[:, :, i:], 0.0)

    dx = sum(s["w"][:, None, :, i] * ahead(i) for i in range(W))
    return {"dx": dx.to(s["x"].dtype), "dw": dw, "dbias": dy.sum(2).sum(0)}


def _plain_conv_step(s):
    x = s["x"].float()
    y = s["w"][..., 0] * x + (s["w"][..., 1:].permute(0, 2, 1) * s["state"]).sum(2) + s["bias"]
    s["state"].copy_(torch.cat([x[:, :, None], s["state"][:, :, :-1]], 2))
    return {"out": (y * torch.sigmoid(y) if s["silu"] else y).to(s["x"].dtype), "state": s["state"]}


def _angles(s, T):
    """cos and sin [B or 1, 1, T, R/2], times rot_scale; the angles in 64 bits."""
    pos = s["positions"] if s["positions"] is not None else torch.arange(T, device=s["q"].device)[None]
    t = pos.double()[:, None, :, None] * s["inv_freq"].double()
    return torch.cos(t).float() * s["rot_scale"], torch.sin(t).float() * s["rot_scale"]


def _turn(s, n, cos, sin):
    R = 2 * s["inv_freq"].numel()
    if s["interleaved"]:
        a, b = n[..., 0:R:2], n[..., 1:R:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = n[..., : R // 2], n[..., R // 2 : R]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, n[..., R:]], -1)


def _rms(x):
    return torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _plain_rot(s):
    cos, sin = _angles(s, s["q"].shape[2])

    def one(x, w):
        n = x.float()
        return _turn(s, n * _rms(n) * w if s["norm"] else n, cos, sin).to(x.dtype)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _plain_rot_bwd(s):
    cos, sin = _angles(s, s["q"].shape[2])
    r = {}

    def one(x, w, dout, name):
        dn, dt = _turn(s, dout.float(), cos, -sin), x.dtype
        if s["norm"]:
            x = x.float()
            f = _rms(x)
            xn = x * f
            r["dw" + name] = (dn * xn).sum(2).sum((0, 1))
            d = dn * w
            dn = f * (d - xn * ((d * xn).sum(-1, keepdim=True) / x.shape[-1]))
        r["d" + name] = dn.to(dt)

    one(s["q"], s["wq"], s["dq_out"], "q")
    one(s["k"], s["wk"], s["dk_out"], "k")
    return r


# ---- the library's calls ------------------------------------------------------------------------
def _own(s):
    lib, op = s["lib"], s["op"]
    if op in ("fwd", "bwd", "step"):
        scan = (s["q"], s["k"], s["v"], s["dt"], s["A"])
        more = dict(dt_bias=s["dt_bias"], skip=s["skip"])
    if op == "fwd":
        out = lib.mesa_ssm_forward_chunked(*scan, **more, starts=s["starts"], S0=s["S0"], S_final=s["S_final"],
                                           workspace=s["workspace"])
        return {"out": out} if s["S_final"] is None else {"out": out, "S_final": s["S_final"]}
    if op == "bwd":
        r = lib.mesa_ssm_backward_chunked(*scan, s["dout"], **more, starts=s["starts"], workspace=s["workspace"])
        return {k: v for k, v in zip(("dq", "dk", "dv", "ddt", "dA", "ddt_bias", "dskip"), r) if v is not None}
    if op == "step":
        return {"out": lib.mesa_ssm_step(s["S"], *scan, **more), "S": s["S"]}
    if op == "conv":
        return {"out": lib.mesa_causal_conv(s["x"], s["w"], bias=s["bias"], silu=s["silu"], starts=s["starts"])}
    if op == "conv_bwd":
        return dict(zip(("dx", "dw", "dbias"), lib.mesa_causal_conv_backward(
            s["x"], s["w"], s["dout"], bias=s["bias"], silu=s["silu"], starts=s["starts"], workspace=s["workspace"])))
    if op == "conv_step":
        return {"out": lib.mesa_causal_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], silu=s["silu"]),
                "state": s["state"]}
    how = dict(wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"], positions=s["positions"], interleaved=s["interleaved"],
               rot_scale=s["rot_scale"], norm=s["norm"], eps=EPS)
    if op == "rot":
        return dict(zip(("q", "k"), lib.mesa_qk_norm_rotary(s["q"], s["k"], **how)))
    r = lib.mesa_qk_norm_rotary_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], **how, workspace=s["workspace"])
    return {k: v for k, v in zip(("dq", "dk", "dwq", "dwk"), r) if v is not None}


PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "conv": _plain_conv, "conv_bwd": _plain_conv_bwd,
         "conv_step": _plain_conv_step, "rot": _plain_rot, "rot_bwd": _plain_rot_bwd}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------------------
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("fwd", "bwd"):
        B, H, Hk, T, dk, dv = (case[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
        qk, vo, gates = B * Hk * T * dk * esz, B * H * T * dv * esz, 4 * B * H * T
        starts = B * T if case["packed"] else 0
        if op == "fwd":  # q, k, v, dt in, o out; u k^T and S q of each token
            return {"bytes": 2 * qk + 2 * vo + gates + starts + (8 * B * H * dk * dv if case["states"] else 0),
                    "flops": 4.0 * B * H * T * dk * dv}
        # q, k, v, dout, dt in, their gradients out; the states again (2), their adjoints (2), dq, dk, dv from them (6)
        return {"bytes": 4 * qk + 3 * vo + gates + starts + B * H * T * esz, "flops": 10.0 * B * H * T * dk * dv}
    if op == "step":
        N, H, Hk, dk, dv = (case[n] for n in ("N", "H", "Hk", "dk", "dv"))
        return {"bytes": 8 * N * H * dk * dv + esz * (2 * N * Hk * dk + 2 * N * H * dv) + 4 * N * H,
                "flops": 4.0 * N * H * dk * dv}
    if op in ("conv", "conv_bwd", "conv_step"):
        B, H, T, d, W = (case[n] for n in ("B", "H", "T", "d", "W"))
        n, weights, starts = B * H * T * d, 4 * H * d * (W + 1), B * T if case["packed"] else 0
        if op == "conv":
            return {"bytes": 2 * n * esz + weights + starts, "flops": 2.0 * n * W}
        if op == "conv_bwd":
            return {"bytes": 3 * n * esz + 2 * weights + starts, "flops": 6.0 * n * W}
        return {"bytes": 2 * n * esz + 8 * n * (W - 1) + weights, "flops": 2.0 * n * W}
    B, H, Hk, T, d = (case[n] for n in ("B", "H", "Hk", "T", "d"))
    n = B * (H + Hk) * T * d
    more = (4 * B * T if case["far"] else 0) + 2 * case["R"] + (8 * d if case["norm"] else 0)
    if op == "rot":
        return {"bytes": 2 * n * esz + more, "flops": 8.0 * n}
    return {"bytes": (3 if case["norm"] else 2) * n * esz + more + (8 * d if case["norm"] else 0), "flops": 16.0 * n}


# ---- the definitions in 64 bits -------------------------------------------------------------------
def _exact_scan(s, op):
    B, H, T = s["dt"].shape
    U, group, dv = B * H, H // s["q"].shape[1], s["v"].shape[-1]

    def seq(x, shared=False):  # token-major [T, U, .]
        x = x.double()
        if shared:
            x = x.repeat_interleave(group, dim=1)
        return x.reshape(U, T, -1).transpose(0, 1).contiguous()

    q, k, v = seq(s["q"], True), seq(s["k"], True), seq(s["v"])
    dk = k.shape[-1]
    raw = s["dt"].double() + s["dt_bias"].double()[:, None]
    step = seq(torch.logaddexp(raw, torch.zeros_like(raw))[..., None])
    A = s["A"].double().repeat(B)[:, None]
    skip = s["skip"].double().repeat(B)[:, None] if s["skip"] is not None else torch.zeros_like(A)
    a = torch.exp(step * A)
    if s["starts"] is not None:
        a = torch.where(s["starts"][:, None].expand(B, H, T).reshape(U, T).t()[..., None], 0.0, a)
    u = step * v
    S = s["S0"].double().reshape(U, dv, dk).clone() if s["S0"] is not None else v.new_zeros((U, dv, dk))
    if op == "fwd":
        out = torch.empty_like(v)
        for t in range(T):
            S.mul_(a[t][..., None]).baddbmm_(u[t][..., None], k[t][:, None, :])
            torch.add(torch.bmm(S, q[t][..., None])[..., 0], skip * v[t], out=out[t])
        r = {"out": out.transpose(0, 1).reshape(B, H, T, dv)}
        if s["S_final"] is not None:
            r["S_final"] = S.view(B, H, dv, dk)
        return r
    g, span, saved = seq(s["dout"]), 32, []
    for t in range(T):
        if t % span == 0:
            saved.append(S.clone())
        S.mul_(a[t][..., None]).baddbmm_(u[t][..., None], k[t][:, None, :])
    dq, dk_, du, da = (torch.empty_like(x) for x in (q, k, v, a))
    R = torch.zeros_like(S)  # adjoint of S_t, of the tokens after t at first
    for start in range((T - 1) // span * span, -1, -span):
        states = [saved[start // span]]
        for t in range(start, min(T, start + span)):
            states.append((states[-1] * a[t][..., None]).baddbmm_(u[t][..., None], k[t][:, None, :]))
        for t in range(min(T, start + span) - 1, start - 1, -1):
            before, after = states[t - start], states[t - start + 1]
            dq[t] = (after.mT @ g[t][..., None])[..., 0]
            R.baddbmm_(g[t][..., None], q[t][:, None, :])
            du[t] = (R @ k[t][..., None])[..., 0]
            dk_[t] = (R.mT @ u[t][..., None])[..., 0]
            da[t] = a[t] * (R * before).sum((-1, -2))[:, None]  # d log a
            R.mul_(a[t][..., None])
    dstep = (du * v).sum(-1, keepdim=True) + A * da
    draw_ = dstep * torch.sigmoid(seq(raw[..., None]))

    def back(x, shared=False):
        x = x.transpose(0, 1).reshape(B, H, T, -1)
        return x.view(B, H // group, group, T, x.shape[-1]).sum(2) if shared else x

    draw_ = back(draw_)[..., 0]
    r = {"dq": back(dq, True), "dk": back(dk_, True), "dv": back(step * du + skip * g), "ddt": draw_,
         "dA": back(step * da)[..., 0].sum((0, 2)), "ddt_bias": draw_.sum((0, 2))}
    if s["skip"] is not None:
        r["dskip"] = back(g * v).sum((0, 2, 3))
    return r


def _exact_conv(s, op):
    t = {n: s[n].double().requires_grad_(op == "conv_bwd") for n in ("x", "w", "bias")}
    x, w, W = t["x"], t["w"], s["w"].shape[-1]
    if op == "conv_step":
        past = torch.cat([x[:, :, None], s["state"].double()], 2)  # [N, H, W, d]
        y = torch.einsum("nhsd,hds->nhd", past, w) + t["bias"]
        return {"out": y * torch.sigmoid(y) if s["silu"] else y, "state": past[:, :, :-1]}
    T = x.shape[2]
    at = torch.arange(T, device=x.device)
    start = torch.zeros((x.shape[0], T), dtype=torch.long, device=x.device)
    if s["starts"] is not None:  # each token's document begins at
        start = torch.where(s["starts"], at, 0).cummax(-1).values
    y = t["bias"][:, None].expand_as(x)
    for i in range(min(W, T)):
        keep = (at - i >= start)[:, None, i:, None]
        y = y + torch.nn.functional.pad(x[:, :, : T - i] * keep * w[:, None, :, i], (0, 0, i, 0))
    out = y * torch.sigmoid(y) if s["silu"] else y
    if op == "conv":
        return {"out": out}
    return {"d" + n: g for n, g in zip(t, torch.autograd.grad((out * s["dout"].double()).sum(), list(t.values())))}


def _exact_rot(s, op):
    T, f = s["q"].shape[2], s["inv_freq"].double()
    pos = s["positions"].double()[:, None] if s["positions"] is not None else torch.arange(
        T, device=f.device, dtype=torch.float64)[None, None]
    turn = s["rot_scale"] * torch.polar(torch.ones_like(pos[..., None] * f), pos[..., None] * f)
    R = 2 * f.numel()
    names = ["q", "k"] + (["wq", "wk"] if s["norm"] else [])
    t = {n: s[n].double().requires_grad_(op == "rot_bwd") for n in names}

    def one(x, w):
        n = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w if w is not None else x
        a, b = (n[..., 0:R:2], n[..., 1:R:2]) if s["interleaved"] else (n[..., : R // 2], n[..., R // 2 : R])
        c = torch.complex(a, b) * turn
        r = torch.view_as_real(c).flatten(-2) if s["interleaved"] else torch.cat([c.real, c.imag], -1)
        return torch.cat([r, n[..., R:]], -1)

    q, k = one(t["q"], t.get("wq")), one(t["k"], t.get("wk"))
    if op == "rot":
        return {"q": q, "k": k}
    L = (q * s["dq_out"].double()).sum() + (k * s["dk_out"].double()).sum()
    return {"d" + n: g for n, g in zip(t, torch.autograd.grad(L, list(t.values())))}


def exact(case, seed):
    op = case["op"]
    if op == "bwd" and case["T"] > 32768:  # a token at a time: too long
        return None
    s = prepare(case, seed)
    if op in ("fwd", "bwd"):
        if op == "bwd":
            s["S0"] = None
        return _exact_scan(s, op)
    if op in ("conv", "conv_bwd", "conv_step"):
        return _exact_conv(s, op)
    if op in ("rot", "rot_bwd"):
        return _exact_rot(s, op)
    group = case["H"] // case["Hk"]
    q, k = (x.double().repeat_interleave(group, dim=1) for x in (s["q"], s["k"]))
    raw = s["dt"].double() + s["dt_bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    S = s["S"].double() * torch.exp(step * s["A"].double())[..., None, None]
    S = S + torch.einsum("nh,nhv,nhk->nhvk", step, s["v"].double(), k)
    out = torch.einsum("nhvk,nhk->nhv", S, q)
    if s["skip"] is not None:
        out = out + s["skip"].double()[:, None] * s["v"].double()
    return {"out": out, "S": S}
