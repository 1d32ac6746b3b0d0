"""A small decoder of gated delta rule blocks: trained a few steps, then decoded token by token.

    python examples/delta_block.py [--steps N] [--dtype bf16|f32]

Each block reads h = rmsnorm(x), projects it to queries, values, an output gate and the two gates
of the recurrence, and the h of the token before to keys (a token is kept under what came before it), runs the gated delta rule, norms and gates each head's
output, and adds its projection to the residual stream; the norm of the next block's input is
part of the same call.  Training differentiates through mesa_delta_backward_chunked and
mesa_block_norm_backward; decoding keeps one state per head and calls mesa_delta_step.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mesa_layer_gb300 import binding  # noqa: E402


class GatedDelta(torch.autograd.Function):
    """out, S_final of the gated delta rule; q, k [B, Hk, T, dk], v [B, H, T, dv]."""

    @staticmethod
    def forward(ctx, q, k, v, gamma, beta, scale):
        out = binding.mesa_delta_forward_chunked(q, k, v, gamma, beta, scale)
        ctx.save_for_backward(q, k, v, gamma, beta)
        ctx.scale = scale
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, gamma, beta = ctx.saved_tensors
        dq, dk, dv, dgamma, dbeta = binding.mesa_delta_backward_chunked(q, k, v, gamma, beta, dout.contiguous(), ctx.scale,
                                                                       gates_dtype=gamma.dtype)
        return dq, dk, dv, dgamma, dbeta, None


class BlockNorm(torch.autograd.Function):
    """x', h of mesa_block_norm (h None without w_pre)."""

    @staticmethod
    def forward(ctx, x, y, gate, w_post, res_scale, w_pre, eps):
        ctx.save_for_backward(x, y, gate, w_post, res_scale, w_pre)
        ctx.eps = eps
        return binding.mesa_block_norm(x, y, gate, w_post, res_scale, w_pre, eps)

    @staticmethod
    def backward(ctx, dx_out, dh):
        x, y, gate, w_post, res_scale, w_pre = ctx.saved_tensors
        dx_out, dh = (None if t is None else t.contiguous() for t in (dx_out, dh))
        return (*binding.mesa_block_norm_backward(x, y, dx_out, dh, gate, w_post, res_scale, w_pre, ctx.eps), None)


def block_norm(x, y, gate=None, w_post=None, res_scale=None, w_pre=None, eps=1e-6):
    return BlockNorm.apply(x, y, gate, w_post, res_scale, w_pre, eps)


class Decoder:
    """`layers` blocks of H heads (Hk of them with queries and keys of their own) of d channels."""

    def __init__(self, vocab=64, layers=2, H=4, Hk=2, d=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.Hk, self.d, self.dtype, self.layers = H, Hk, d, dtype, layers
        D = self.D = H * d

        def weight(n, m):
            return torch.randn((n, m), generator=g, device="cuda").mul_(n ** -0.5).requires_grad_()

        def ones(n):
            return torch.ones(n, device="cuda", requires_grad=True)

        self.embed = torch.randn((vocab, D), generator=g, device="cuda").requires_grad_()
        self.head = weight(D, vocab)
        self.first = ones(D)  # the first block's input norm
        self.blocks = [dict(q=weight(D, Hk * d), k=weight(D, Hk * d), v=weight(D, D), gate=weight(D, D), ab=weight(D, 2 * H), o=weight(D, D),
                            w_head=ones(d), res_scale=ones(D), w_pre=ones(D)) for _ in range(layers)]

    def parameters(self):
        return [self.embed, self.head, self.first, *(p for b in self.blocks for p in b.values())]

    def _inputs(self, b, h, before):
        """h [B, T, D], before (the same, a token earlier) -> q, k, v [B, heads, T, d], gate [B, H, T, d],
        gamma, beta [B, H, T]."""
        B, T, _ = h.shape

        def heads(x, n):
            return x.view(B, T, n, -1).transpose(1, 2)

        q, k = (F.normalize(heads(t @ b[n].to(h.dtype), self.Hk).float(), dim=-1, eps=1e-6).to(h.dtype)
                for t, n in ((h, "q"), (before, "k")))
        a, beta = heads(h.float() @ b["ab"], 2 * self.H)[..., 0].chunk(2, 1)
        return (q.contiguous(), k.contiguous(), heads(h @ b["v"].to(h.dtype), self.H).contiguous(),
                heads(h @ b["gate"].to(h.dtype), self.H).contiguous(), torch.sigmoid(a + 4.0).contiguous(),
                torch.sigmoid(beta).contiguous())

    def _run(self, tokens, mix, last=None):
        """mix(layer, q, k, v, gamma, beta) -> out; logits of every token.  last: each layer's h of the
        token before the first (zero without), replaced with that of the last one."""
        x = self.embed[tokens].to(self.dtype)
        x, h = block_norm(None, x, w_pre=self.first)
        for i, b in enumerate(self.blocks):
            first = torch.zeros_like(h[:, :1]) if last is None or last[i] is None else last[i]
            q, k, v, gate, gamma, beta = self._inputs(b, h, torch.cat((first, h[:, :-1]), 1))
            if last is not None:
                last[i] = h[:, -1:]
            o = mix(i, q, k, v, gamma, beta)
            o, _ = block_norm(None, o, gate, w_post=b["w_head"])  # each head's output, normed and gated
            y = o.transpose(1, 2).reshape(x.shape) @ b["o"].to(self.dtype)
            x, h = block_norm(x, y, res_scale=b["res_scale"], w_pre=b["w_pre"])
        return h.float() @ self.head

    def __call__(self, tokens):
        return self._run(tokens, lambda i, *a: GatedDelta.apply(*a, self.d ** -0.5))

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits and (the states, each layer's last h) after the prompt."""
        B, last = tokens.shape[0], [None] * self.layers
        states = [torch.empty((B, self.H, self.d, self.d), device="cuda") for _ in self.blocks]
        return self._run(tokens, lambda i, *a: binding.mesa_delta_forward_chunked(*a, self.d ** -0.5,
                                                                                 S_final=states[i]), last), (states, last)

    @torch.no_grad()
    def step(self, memory, token):
        """Logits after one more token [B]; the memory that prefill gave is updated in place."""
        states, last = memory

        def mix(i, q, k, v, gamma, beta):
            q, k, v = (t[:, :, 0].contiguous() for t in (q, k, v))
            return binding.mesa_delta_step(states[i], q, k, v, gamma[..., 0].contiguous(), beta[..., 0].contiguous(),
                                           self.d ** -0.5)[:, :, None].contiguous()
        return self._run(token[:, None], mix, last)[:, 0]


def recall_batch(B, T, vocab, seed):
    """Pairs (a, b) drawn from a table of each sequence: after a is seen again, b follows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randint(vocab // 2, vocab, (B, vocab // 2), generator=g, device="cuda")
    a = torch.randint(0, vocab // 2, (B, T // 2), generator=g, device="cuda")
    return torch.stack((a, table.gather(1, a)), -1).view(B, -1)


def train(model, steps, B=8, T=256, vocab=64, lr=2e-3):
    """Adam on the answers' cross-entropy; the loss of every step."""
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for s in range(steps):
        x = recall_batch(B, T, vocab, s)
        logits = model(x)
        loss = F.cross_entropy(logits[:, 0::2].flatten(0, 1), x[:, 1::2].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    args = ap.parse_args()
    model = Decoder(dtype=torch.bfloat16 if args.dtype == "bf16" else torch.float32)
    losses = train(model, args.steps)
    print("loss %.3f -> %.3f in %d steps" % (losses[0], losses[-1], args.steps))
    x = recall_batch(4, 256, 64, 10 ** 6)
    with torch.no_grad():
        whole = model(x)
    _, memory = model.prefill(x[:, :200])
    right = total = 0
    gap = 0.0
    for t in range(200, 256):
        logits = model.step(memory, x[:, t])
        gap = max(gap, float((logits - whole[:, t]).norm() / whole[:, t].norm()))
        if t % 2 == 0:
            right += int((logits.argmax(-1) == x[:, t + 1]).sum())
            total += x.shape[0]
    print("decoded %d answers, %d right; step logits against the whole sequence's: %.1e" % (total, right, gap))


if __name__ == "__main__":
    main()
