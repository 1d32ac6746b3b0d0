"""A small decoder of selective scan blocks: trained a few steps, then decoded token by token.

    python examples/scan_block.py [--steps N] [--dtype bf16|f32]

Each block projects h = rmsnorm(x) to values, queries, keys, an output gate and step lengths, runs a short causal
convolution with SiLU over values, queries and keys, norms and rotates queries and keys per head, runs the selective
scan, norms and gates each head's output, and adds its projection to the residual stream; the norm of the next block's
input is part of the same call.  Training differentiates through the library's backward calls (documents may be packed
into one row); decoding keeps a window of inputs and a state per head.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]
from delta_block import block_norm, recall_batch, train  # noqa: E402
from mesa_layer_gb300 import binding  # noqa: E402


class CausalConv(torch.autograd.Function):
    """silu(conv(x)) over time; x [B, H, T, d], w [H, d, W], bias [H, d], starts [B, T] or None."""

    @staticmethod
    def forward(ctx, x, w, bias, starts):
        ctx.save_for_backward(x, w, bias)
        ctx.starts = starts
        return binding.mesa_causal_conv(x, w, bias=bias, starts=starts)

    @staticmethod
    def backward(ctx, dout):
        x, w, bias = ctx.saved_tensors
        return (*binding.mesa_causal_conv_backward(x, w, dout.contiguous(), bias=bias, starts=ctx.starts), None)


class NormRotary(torch.autograd.Function):
    """Per-head norm and position rotation of q [B, H, T, d] and k [B, Hk, T, d]."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, inv_freq, positions):
        ctx.save_for_backward(q, k, wq, wk, inv_freq)
        ctx.positions = positions
        return binding.mesa_qk_norm_rotary(q, k, wq, wk, inv_freq, positions=positions)

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, inv_freq = ctx.saved_tensors
        return (*binding.mesa_qk_norm_rotary_backward(q, k, dq_out.contiguous(), dk_out.contiguous(), wq, wk, inv_freq,
                                                      positions=ctx.positions), None, None)


class Scan(torch.autograd.Function):
    """The selective scan of q, k [B, Hk, T, dk], v [B, H, T, dv], steps dt [B, H, T]."""

    @staticmethod
    def forward(ctx, q, k, v, dt, A, dt_bias, skip, starts):
        ctx.save_for_backward(q, k, v, dt, A, dt_bias, skip)
        ctx.starts = starts
        return binding.mesa_ssm_forward_chunked(q, k, v, dt, A, dt_bias, skip, starts)

    @staticmethod
    def backward(ctx, dout):
        q, k, v, dt, A, dt_bias, skip = ctx.saved_tensors
        return (*binding.mesa_ssm_backward_chunked(q, k, v, dt, A, dout.contiguous(), dt_bias, skip, ctx.starts,
                                                   gates_dtype=torch.float32), None)


class Decoder:
    """`layers` blocks of H heads (Hk of them with queries and keys of their own) of d channels."""

    def __init__(self, vocab=64, layers=2, H=4, Hk=2, d=128, W=4, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.Hk, self.d, self.W, self.dtype, self.layers = H, Hk, d, W, dtype, layers
        D, rows = H * d, H + 2 * Hk

        def weight(n, m):
            return torch.randn((n, m), generator=g, device="cuda").mul_(n ** -0.5).requires_grad_()

        def full(x, *n):
            return torch.full(n, x, device="cuda").requires_grad_()

        self.embed = torch.randn((vocab, D), generator=g, device="cuda").requires_grad_()
        self.head = weight(D, vocab)
        self.first = full(1.0, D)  # the first block's input norm
        self.inv_freq = torch.tensor([10000.0 ** (-4.0 * j / d) for j in range(d // 4)], device="cuda")  # half of the channels
        self.blocks = [dict(vqk=weight(D, rows * d), gate=weight(D, D), dt=weight(D, H), o=weight(D, D),
                            taps=(torch.randn((rows, d, W), generator=g, device="cuda") * W ** -0.5).requires_grad_(),
                            bias=full(0.0, rows, d), wq=full(d ** -0.5, d), wk=full(1.0, d),
                            log_A=torch.linspace(0.0, 2.0, H, device="cuda").requires_grad_(), dt_bias=full(-3.0, H), skip=full(1.0, H),
                            w_head=full(1.0, d), res_scale=full(1.0, D), w_pre=full(1.0, D)) for _ in range(layers)]

    def parameters(self):
        return [self.embed, self.head, self.first, *(p for b in self.blocks for p in b.values())]

    def _run(self, tokens, conv, rotary, scan):
        """conv(layer, b, x), rotary(layer, b, q, k), scan(layer, b, q, k, v, dt, A); logits of every token."""
        B, T = tokens.shape

        def heads(x, n):
            return x.view(B, T, n, -1).transpose(1, 2).contiguous()

        x = self.embed[tokens].to(self.dtype)
        x, h = block_norm(None, x, w_pre=self.first)
        for i, b in enumerate(self.blocks):
            vqk = conv(i, b, heads(h @ b["vqk"].to(h.dtype), self.H + 2 * self.Hk))
            v, q, k = (t.contiguous() for t in vqk.split((self.H, self.Hk, self.Hk), 1))
            q, k = rotary(i, b, q, k)
            o = scan(i, b, q, k, v, heads(h.float() @ b["dt"], self.H)[..., 0].contiguous(), -torch.exp(b["log_A"]))
            o, _ = block_norm(None, o, heads(h @ b["gate"].to(h.dtype), self.H), w_post=b["w_head"])
            y = o.transpose(1, 2).reshape(x.shape) @ b["o"].to(self.dtype)
            x, h = block_norm(x, y, res_scale=b["res_scale"], w_pre=b["w_pre"])
        return h.float() @ self.head

    def __call__(self, tokens, starts=None):
        """Logits; starts [B, T] marks the first tokens of documents packed into a row."""
        positions = None
        if starts is not None:  # each document counts its own
            at = torch.arange(tokens.shape[1], device="cuda").expand(tokens.shape)
            positions = (at - torch.where(starts, at, 0).cummax(-1).values).to(torch.int32)
        return self._run(tokens, lambda i, b, x: CausalConv.apply(x, b["taps"], b["bias"], starts),
                         lambda i, b, q, k: NormRotary.apply(q, k, b["wq"], b["wk"], self.inv_freq, positions),
                         lambda i, b, q, k, v, dt, A: Scan.apply(q, k, v, dt, A, b["dt_bias"], b["skip"], starts))

    @torch.no_grad()
    def prefill(self, tokens):
        """Logits and the memory after the prompt: windows, states, the next position."""
        B, rows = tokens.shape[0], self.H + 2 * self.Hk
        windows = [torch.empty((B, rows, self.W - 1, self.d), device="cuda") for _ in self.blocks]
        states = [torch.empty((B, self.H, self.d, self.d), device="cuda") for _ in self.blocks]
        logits = self._run(
            tokens, lambda i, b, x: binding.mesa_causal_conv(x, b["taps"], bias=b["bias"], state_final=windows[i]),
            lambda i, b, q, k: binding.mesa_qk_norm_rotary(q, k, b["wq"], b["wk"], self.inv_freq),
            lambda i, b, *a: binding.mesa_ssm_forward_chunked(*a, b["dt_bias"], b["skip"], S_final=states[i]))
        return logits, [windows, states, tokens.shape[1]]

    @torch.no_grad()
    def step(self, memory, token):
        """Logits after one more token [B]; the memory that prefill gave is updated in place."""
        windows, states, at = memory
        memory[2] += 1

        def conv(i, b, x):
            return binding.mesa_causal_conv_step(x[:, :, 0].contiguous(), b["taps"], windows[i], bias=b["bias"])[:, :, None]

        def scan(i, b, q, k, v, dt, A):
            q, k, v, dt = (t[:, :, 0].contiguous() for t in (q, k, v, dt))
            return binding.mesa_ssm_step(states[i], q, k, v, dt, A, b["dt_bias"], b["skip"])[:, :, None].contiguous()

        return self._run(token[:, None], conv,
                         lambda i, b, q, k: binding.mesa_qk_norm_rotary(q, k, b["wq"], b["wk"], self.inv_freq, offset=at), scan)[:, 0]


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
