"""The selective scan in 64 bits, 64 tokens at once, for sequences that a token recurrence takes too long for; autograd takes
the gradients from it, those of the tokens' log-decays among them."""
import torch


def chunked(q, k, v, dt, A, dt_bias=None, skip=None, starts=None, S0=None, C=64):
    """(out, S_final, log a) of q, k [B, Hk, T, dk], v [B, H, T, dv], dt [B, H, T], A, dt_bias, skip [H], starts [B, T]."""
    B, H, T, dv = v.shape
    q, k = (x.repeat_interleave(H // q.shape[1], dim=1) for x in (q, k))
    raw = dt if dt_bias is None else dt + dt_bias[:, None]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    log = step * A[:, None]  # (a document's first token forgets all, whatever its step: told by `document`)
    if log.requires_grad:
        log.retain_grad()
    S = torch.zeros(B, H, dv, q.shape[-1], dtype=v.dtype, device=v.device) if S0 is None else S0
    document = torch.zeros(B, T, dtype=torch.long, device=v.device) if starts is None else starts.long().cumsum(-1)
    before, out = torch.zeros(B, dtype=torch.long, device=v.device), []
    for t in range(0, T, C):
        e = slice(t, min(t + C, T))
        d = document[:, None, e]
        # log[t] counts between writers before t and readers from t on: not where t is its document's first
        first = torch.zeros_like(d, dtype=torch.bool) if starts is None else starts[:, None, e]
        c = torch.where(first, torch.zeros_like(log[:, :, e]), log[:, :, e]).cumsum(-1)
        n = c.shape[-1]
        low = torch.ones(n, n, device=v.device).tril().bool() & (d[..., :, None] == d[..., None, :])
        M = torch.exp(torch.where(low, c[..., :, None] - c[..., None, :], -torch.inf)) * step[:, :, None, e]
        into = torch.exp(torch.where(d == before[:, None, None], c, -torch.inf))
        last = torch.exp(torch.where(d == d[..., -1:], c[..., -1:] - c, -torch.inf)) * step[:, :, e]
        out.append(into[..., None] * (q[:, :, e] @ S.mT) + ((q[:, :, e] @ k[:, :, e].mT) * M) @ v[:, :, e])
        S = into[..., -1, None, None] * S + (last[..., None] * v[:, :, e]).mT @ k[:, :, e]
        before = d[:, 0, -1]
    out = torch.cat(out, 2)
    return out if skip is None else out + skip[:, None, None] * v, S, log


def gradients(s):
    """Gradients in 64 bits of a case's inputs for dout and dS_final, by name, and "log", those of its log-decays."""
    x = {n: None if s[n] is None else s[n].double().requires_grad_() for n in ("q", "k", "v", "dt", "A", "dt_bias", "skip", "S0")}
    out, S, log = chunked(x["q"], x["k"], x["v"], x["dt"], x["A"], x["dt_bias"], x["skip"], s["starts"], x["S0"])
    L = (out * s["dout"].double()).sum()
    if s["dS_final"] is not None:
        L = L + (S * s["dS_final"].double()).sum()
    L.backward()
    return {"log": log.grad, **{n: t.grad for n, t in x.items() if t is not None}}


def chunks_shares(x, L=128):
    """Sums over 128 tokens each of x [B, H, T]."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % L)).unflatten(-1, (-1, L)).sum(-1)
