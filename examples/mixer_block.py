"""A gated-delta-rule block from this library's operators, as a user runs it.

    norm -> q, k, v projections -> causal depthwise conv + SiLU -> unit-length q, k
         -> gated delta rule -> norm of each head -> output projection (+ residual)

Prefill runs whole sequences and leaves two states per layer, the convolution's
last K-1 inputs and the delta rule's matrix; decoding advances both one token
at a time; a training step takes the same block backwards.  The projections are
plain matrix products of the framework; everything else on the path is this
library's (the unit length of q and k and the gates are elementwise).

    python examples/mixer_block.py          # prefill, decode, a few training steps; prints what it saw
    python examples/mixer_block.py --time gdr_bwd --batch 2 --tokens 2048 --key-heads 16 --value-heads 32
                                            # one operator alone: gdr_fwd, gdr_bwd, gdr_step, ln_fwd, ln_bwd
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402


class Block:
    def __init__(self, dim: int, key_heads: int, value_heads: int, head: int, width: int = 4, dtype=torch.bfloat16,
                 seed: int = 0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s, scale: (torch.randn(s, generator=gen) * scale).to(dtype).to(device)  # noqa: E731
        self.hk, self.hv, self.d = key_heads, value_heads, head
        self.channels = (2 * key_heads + value_heads) * head
        self.norm = (torch.ones(dim, device=device), torch.zeros(dim, device=device))
        self.head_norm = (torch.ones(head, device=device), torch.zeros(head, device=device))
        self.w_in = rnd(self.channels, dim, scale=dim ** -0.5)
        self.w_gate = rnd(2 * value_heads, dim, scale=dim ** -0.5)
        self.w_out = rnd(dim, value_heads * head, scale=(value_heads * head) ** -0.5)
        self.conv = rnd(self.channels, width, scale=0.4)
        self.rate = torch.rand(value_heads, generator=gen).to(device) * 2 + 0.05
        self.params = [self.w_in, self.w_gate, self.w_out, self.conv]

    def _split(self, y):
        """Channels [B, L, C] to q, k [B,L,Hk,D] of unit length and v [B,L,Hv,D]."""
        n = self.hk * self.d
        q, k, v = y[..., :n], y[..., n:2 * n], y[..., 2 * n:]
        unit = lambda x: F.normalize(x.unflatten(-1, (self.hk, self.d)).float(), dim=-1).to(x.dtype)  # noqa: E731
        return unit(q), unit(k), v.unflatten(-1, (self.hv, self.d))

    def _gates(self, h):
        a, b = F.linear(h, self.w_gate).chunk(2, -1)
        return (-self.rate * F.softplus(a.float())).contiguous(), torch.sigmoid(b).contiguous()

    def _out(self, x, o):
        o = ccv.layer_norm_fwd(o, *self.head_norm)
        return x + F.linear(o.flatten(-2), self.w_out)

    def prefill(self, x, seq_idx=None):
        """x [B, L, dim] -> (output, states); the convolution reads the channel-last projection as it lies."""
        h = ccv.layer_norm_fwd(x, *self.norm)
        z = F.linear(h, self.w_in)
        y, conv_state = ccv.causal_conv1d_fwd(z.transpose(1, 2), self.conv, activation="silu", seq_idx=seq_idx,
                                              return_final_states=True)
        q, k, v = self._split(y.transpose(1, 2))
        g, beta = self._gates(h)
        o, state = ccv.gated_delta_rule_fwd(q, k, v, g, beta, seq_idx=seq_idx, return_final_state=True)
        return self._out(x, o), (conv_state.contiguous(), state)

    def decode(self, x, states):
        """x [B, dim], one token; the states are advanced in place."""
        conv_state, state = states
        h = ccv.layer_norm_fwd(x, *self.norm)
        y = ccv.causal_conv1d_update(F.linear(h, self.w_in), conv_state, self.conv, activation="silu")
        q, k, v = (t.squeeze(1) for t in self._split(y.unsqueeze(1)))
        g, beta = self._gates(h)
        return self._out(x, ccv.gated_delta_rule_step(q, k, v, g, beta, state))


class DeltaRule(torch.autograd.Function):
    """The delta rule as a function of a training graph."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, seq_idx):
        ctx.save_for_backward(q, k, v, g, beta)
        ctx.seq_idx = seq_idx
        return ccv.gated_delta_rule_fwd(q, k, v, g, beta, seq_idx=seq_idx)

    @staticmethod
    def backward(ctx, dout):
        return ccv.gated_delta_rule_bwd(*ctx.saved_tensors, dout, seq_idx=ctx.seq_idx)[:5] + (None,)


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return ccv.layer_norm_fwd(x, weight, bias)

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias = ctx.saved_tensors
        return ccv.layer_norm_bwd(x, weight, dout.contiguous(), bias)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, seq_idx):
        ctx.save_for_backward(x, weight)
        ctx.seq_idx = seq_idx
        return ccv.causal_conv1d_fwd(x, weight, activation="silu", seq_idx=seq_idx)

    @staticmethod
    def backward(ctx, dout):
        x, weight = ctx.saved_tensors
        dx, dw, _, _ = ccv.causal_conv1d_bwd(x, weight, dout, activation="silu", seq_idx=ctx.seq_idx)
        return dx, dw, None


def training_loss(block: Block, x, target, seq_idx=None):
    """The block's output through functions that know their gradients."""
    h = LayerNorm.apply(x, *block.norm)
    y = Conv.apply(F.linear(h, block.w_in).transpose(1, 2), block.conv, seq_idx)
    q, k, v = block._split(y.transpose(1, 2))
    g, beta = block._gates(h)
    o = LayerNorm.apply(DeltaRule.apply(q, k, v, g, beta, seq_idx), *block.head_norm)
    out = x + F.linear(o.flatten(-2), block.w_out)
    return ((out.float() - target) ** 2).mean()


def train_step(block: Block, x, target, seq_idx=None, lr: float = 0.0):
    leaves = block.params + list(block.norm) + list(block.head_norm)
    for p in leaves:
        p.requires_grad_(True)
        p.grad = None
    loss = training_loss(block, x, target, seq_idx)
    loss.backward()
    grads = [p.grad for p in leaves]
    with torch.no_grad():
        for p in leaves:
            p.requires_grad_(False)
            p -= lr * p.grad.to(p.dtype)
    return loss.detach(), grads


def time_operator(name: str, batch: int, tokens: int, key_heads: int, value_heads: int, head: int, steps: int):
    """Microseconds of one call of an operator on bf16 data of these sizes, calls back to back on the device."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    T = 1 if name == "gdr_step" else tokens
    q, k = (F.normalize(rnd(batch, T, key_heads, head), dim=-1).bfloat16() for _ in range(2))
    v, dout = (rnd(batch, T, value_heads, head).bfloat16() for _ in range(2))
    g, beta = -F.softplus(rnd(batch, T, value_heads)), torch.sigmoid(rnd(batch, T, value_heads)).bfloat16()
    state = rnd(batch, value_heads, head, head)
    x, w = v.reshape(batch * T, -1), torch.ones(value_heads * head, device="cuda").bfloat16()
    call = {"gdr_fwd": lambda: ccv.gated_delta_rule_fwd(q, k, v, g, beta, return_final_state=True),
            "gdr_bwd": lambda: ccv.gated_delta_rule_bwd(q, k, v, g, beta, dout),
            "gdr_step": lambda: ccv.gated_delta_rule_step(q, k, v, g, beta, state),
            "ln_fwd": lambda: ccv.layer_norm_fwd(x, w, w),
            "ln_bwd": lambda: ccv.layer_norm_bwd(x, w, dout.reshape(x.shape), w)}[name]
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        call()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / steps * 1e3


def main(argv=None):
    ap = argparse.ArgumentParser(description="The block's operators together, or one of them timed.")
    ap.add_argument("--time", choices=("gdr_fwd", "gdr_bwd", "gdr_step", "ln_fwd", "ln_bwd"))
    for flag, n in (("batch", 2), ("tokens", 2048), ("key-heads", 16), ("value-heads", 32), ("head", 128),
                    ("steps", 20)):
        ap.add_argument("--" + flag, type=int, default=n)
    a = ap.parse_args(argv)
    if a.time:
        us = time_operator(a.time, a.batch, a.tokens, a.key_heads, a.value_heads, a.head, a.steps)
        print(f"{a.time}: {us:.1f} us")
        return
    block = Block(dim=256, key_heads=2, value_heads=4, head=64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, 160, 256), generator=gen, device="cuda").to(torch.bfloat16)
    whole, _ = block.prefill(x)
    first, states = block.prefill(x[:, :150].contiguous())
    tail = torch.stack([block.decode(x[:, t], states) for t in range(150, 160)], 1)
    gap = (torch.cat([first, tail], 1).float() - whole.float()).abs().max().item()
    print(f"prefill of 160 tokens against prefill of 150 and ten decode steps: largest difference {gap:.4f}")
    target = torch.randn((2, 160, 256), generator=gen, device="cuda")
    losses = [train_step(block, x, target, lr=0.5)[0].item() for _ in range(8)]
    print("training loss", " ".join(f"{v:.4f}" for v in losses))


if __name__ == "__main__":
    main()
