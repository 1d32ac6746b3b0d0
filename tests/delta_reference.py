"""64-bit restatements (numpy, a token at a time) of the gated delta rule, its gradients and the
block norm, and the inputs of their tests."""
import numpy as np

from mesa_layer_gb300.synth import round_bf16


def rule_forward(q, k, v, gamma, beta, scale, S0=None):
    """q, k [B, Hk, T, dk], v [B, H, T, dv], gamma, beta [B, H, T] -> out, S_final (fp64)."""
    q, k, v, gamma, beta = (np.asarray(x, dtype=np.float64) for x in (q, k, v, gamma, beta))
    B, H, T, dv = v.shape
    g = H // q.shape[1] if q.shape[1] else 1
    q, k = q.repeat(g, 1), k.repeat(g, 1)
    S = np.zeros((B, H, dv, q.shape[-1])) if S0 is None else np.array(S0, dtype=np.float64)
    out = np.zeros_like(v)
    for t in range(T):
        S = gamma[:, :, t, None, None] * S
        e = v[:, :, t] - np.einsum("bhvk,bhk->bhv", S, k[:, :, t])
        S = S + np.einsum("bh,bhv,bhk->bhvk", beta[:, :, t], e, k[:, :, t])
        out[:, :, t] = scale * np.einsum("bhvk,bhk->bhv", S, q[:, :, t])
    return out, S


def rule_backward(q, k, v, gamma, beta, scale, dout, S0=None, dS_final=None):
    q, k, v, gamma, beta, dout = (np.asarray(x, dtype=np.float64) for x in (q, k, v, gamma, beta, dout))
    B, H, T, dv = v.shape
    Hk, dk = q.shape[1], q.shape[-1]
    g = H // Hk
    q, k = q.repeat(g, 1), k.repeat(g, 1)
    S = np.zeros((B, H, dv, dk)) if S0 is None else np.array(S0, dtype=np.float64)
    states, es = [S], []
    for t in range(T):
        D = gamma[:, :, t, None, None] * S
        e = v[:, :, t] - np.einsum("bhvk,bhk->bhv", D, k[:, :, t])
        S = D + np.einsum("bh,bhv,bhk->bhvk", beta[:, :, t], e, k[:, :, t])
        states.append(S)
        es.append(e)
    A = np.zeros_like(S) if dS_final is None else np.array(dS_final, dtype=np.float64)
    dq, dk_, dv_, dgamma, dbeta = (np.zeros_like(x) for x in (q, k, v, gamma, beta))
    for t in range(T - 1, -1, -1):
        kt, gt = k[:, :, t], dout[:, :, t]
        dq[:, :, t] = scale * np.einsum("bhvk,bhv->bhk", states[t + 1], gt)
        A = A + scale * np.einsum("bhv,bhk->bhvk", gt, q[:, :, t])
        du = np.einsum("bhvk,bhk->bhv", A, kt)
        dv_[:, :, t] = beta[:, :, t, None] * du
        dbeta[:, :, t] = (du * es[t]).sum(-1)
        dk_[:, :, t] = np.einsum("bhvk,bhv->bhk", A, beta[:, :, t, None] * es[t]) - gamma[:, :, t, None] * np.einsum(
            "bhvk,bhv->bhk", states[t], dv_[:, :, t])
        N = A - np.einsum("bhv,bhk->bhvk", dv_[:, :, t], kt)
        dgamma[:, :, t] = (N * states[t]).sum((-1, -2))
        A = gamma[:, :, t, None, None] * N
    return dict(dq=dq.reshape(B, Hk, g, T, dk).sum(2), dk=dk_.reshape(B, Hk, g, T, dk).sum(2), dv=dv_, dgamma=dgamma,
                dbeta=dbeta, dS0=A)


def rule_inputs(seed, dtype, B, H, Hk, T, dk, dv, gates="open", S0=False):
    """q, k unit rows, v, dout normal.  gates: "open" (0.9 to 1), "wide" (0 to 1), "packed" (closed
    gates and zero betas among open ones), "one" (gamma = 1, beta = 1), "shut" (gamma = 0)."""
    r = np.random.default_rng(seed)
    rnd = round_bf16 if dtype == "bf16" else (lambda x: np.ascontiguousarray(x, dtype=np.float32))

    def unit(shape):
        x = r.standard_normal(shape)
        return x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-12)

    s = dict(q=rnd(unit((B, Hk, T, dk))), k=rnd(unit((B, Hk, T, dk))), v=rnd(r.standard_normal((B, H, T, dv))),
             dout=rnd(r.standard_normal((B, H, T, dv))), gamma=r.uniform(0.9, 1.0, (B, H, T)).astype(np.float32),
             beta=r.uniform(0.0, 1.0, (B, H, T)).astype(np.float32))
    if gates == "wide":
        s["gamma"] = r.uniform(0.0, 1.0, (B, H, T)).astype(np.float32)
        s["beta"] = r.uniform(0.0, 1.8, (B, H, T)).astype(np.float32)
    elif gates == "packed":
        s["gamma"][r.random((B, H, T)) < 0.05] = 0.0
        s["beta"][r.random((B, H, T)) < 0.2] = 0.0
    elif gates == "one":
        s["gamma"][:] = 1.0
        s["beta"][:] = 1.0
    elif gates == "shut":
        s["gamma"][:] = 0.0
    s["S0"] = (0.5 * r.standard_normal((B, H, dv, dk))).astype(np.float32) if S0 else None
    s["dS_final"] = (0.5 * r.standard_normal((B, H, dv, dk))).astype(np.float32) if S0 else None
    return s


def norm_forward(x, y, gate, w_post, res_scale, w_pre, eps):
    y = np.asarray(y, dtype=np.float64)
    z = y if w_post is None else y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w_post
    if gate is not None:
        gate = np.asarray(gate, dtype=np.float64)
        z = z * gate / (1.0 + np.exp(-gate))
    X = z if res_scale is None else res_scale * z
    X = X if x is None else X + np.asarray(x, dtype=np.float64)
    h = None if w_pre is None else X / np.sqrt((X * X).mean(-1, keepdims=True) + eps) * w_pre
    return X, h


def norm_backward(x, y, gate, w_post, res_scale, w_pre, eps, dx_out, dh):
    y = np.asarray(y, dtype=np.float64)
    ry = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if w_post is not None else 1.0
    yh = y * ry
    z = yh * w_post if w_post is not None else yh
    a, da = 1.0, 0.0
    if gate is not None:
        gate = np.asarray(gate, dtype=np.float64)
        s = 1.0 / (1.0 + np.exp(-gate))
        a, da = gate * s, s * (1.0 + gate * (1.0 - s))
    rs = 1.0 if res_scale is None else np.asarray(res_scale, dtype=np.float64)
    X = rs * a * z + (0.0 if x is None else np.asarray(x, dtype=np.float64))
    dX = np.zeros_like(y) if dx_out is None else np.asarray(dx_out, dtype=np.float64)
    r = {}
    if w_pre is not None:
        rx = 1.0 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
        Xh = X * rx
        dh = np.zeros_like(y) if dh is None else np.asarray(dh, dtype=np.float64)
        r["dw_pre"] = (dh * Xh).sum(0)
        d = dh * w_pre
        dX = dX + rx * (d - Xh * (d * Xh).mean(-1, keepdims=True))
    r["dx"] = dX
    r["dres_scale"] = (dX * a * z).sum(0)
    r["dgate"] = dX * rs * z * da
    dz = dX * rs * a
    if w_post is not None:
        r["dw_post"] = (dz * yh).sum(0)
        d = dz * w_post
        r["dy"] = ry * (d - yh * (d * yh).mean(-1, keepdims=True))
    else:
        r["dy"] = dz
    return r
