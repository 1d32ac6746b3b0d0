"""Plain 64-bit forms of the selective scan, the causal convolution and the norm and rotation of queries and keys, token
by token, from which autograd takes the gradients."""
import torch


def scan(q, k, v, dt, A, dt_bias=None, skip=None, starts=None, S0=None):
    """(out, S_final) of q, k [B, Hk, T, dk], v [B, H, T, dv], dt [B, H, T], A, dt_bias, skip [H], starts [B, T]."""
    B, H, T, dv = v.shape
    group = H // q.shape[1]
    q, k = (x.repeat_interleave(group, dim=1) for x in (q, k))
    raw = dt if dt_bias is None else dt + dt_bias[:, None]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    a = torch.exp(step * A[:, None])
    S = torch.zeros(B, H, dv, q.shape[-1], dtype=v.dtype, device=v.device) if S0 is None else S0
    out = []
    for t in range(T):
        if starts is not None:
            S = torch.where(starts[:, t, None, None, None], torch.zeros_like(S), S)
        S = a[:, :, t, None, None] * S + step[:, :, t, None, None] * v[:, :, t, :, None] * k[:, :, t, None, :]
        o = (S * q[:, :, t, None, :]).sum(-1)
        out.append(o if skip is None else o + skip[:, None] * v[:, :, t])
    return (torch.stack(out, 2) if T else v), S


def conv(x, w, bias=None, silu=True, starts=None, state0=None):
    """(out, state after the last token) of x [B, H, T, d], w [H, d, W]."""
    B, H, T, d = x.shape
    W = w.shape[-1]
    past = [torch.zeros(B, H, d, dtype=x.dtype, device=x.device) if state0 is None else state0[:, :, s] for s in range(W - 1)]
    out = []
    for t in range(T):
        if starts is not None:
            past = [torch.where(starts[:, t, None, None], torch.zeros_like(p), p) for p in past]
        past = [x[:, :, t]] + past
        y = sum(w[:, :, s] * past[s] for s in range(W))
        if bias is not None:
            y = y + bias
        out.append(y * torch.sigmoid(y) if silu else y)
        past = past[:W - 1]
    return (torch.stack(out, 2) if T else x), (torch.stack(past, 2) if W > 1 else None)


def rotate(x, w, inv_freq, positions, interleaved, rot_scale, norm, eps):
    """x [B, H, T, d], positions [B, T]."""
    n = x
    if norm:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            n = n * w
    if inv_freq is None:
        return n
    half = inv_freq.numel()
    angle = positions.double()[:, None, :, None] * inv_freq.double()
    c, s = rot_scale * torch.cos(angle), rot_scale * torch.sin(angle)
    out = n.clone()
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[..., i0] = n[..., i0] * c[..., j] - n[..., i1] * s[..., j]
        out[..., i1] = n[..., i1] * c[..., j] + n[..., i0] * s[..., j]
    return out


def off(x, ref):
    """2-norm of the difference over that of the reference (the difference's own where that is zero)."""
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    n = float(ref.norm())
    return float((x - ref).norm()) / (n if n else 1.0)
