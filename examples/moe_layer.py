"""One MoE layer on the dispatcher, trained and then served.

    python examples/moe_layer.py

``train_step`` is a layer's forward and backward pass on one GPU: dispatch, the experts'
gated feed-forward block, combine, and the gradients back through all three. The example
fits the layer to a random target layer for a few steps, quantises the experts to 4 bits
with group scales, and answers a batch of single tokens through ``decode_step``; then to
4-bit floating point, and answers it through the layer for a few tokens, ``moe_layer``.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_topk_ids_expert_gb300 as ep  # noqa: E402


@dataclass
class Experts:
    """bf16 weights the kernels read, fp32 copies the optimiser steps, fp32 gradients."""
    w_gate_up: torch.Tensor   # [E, 2 inter, hidden]
    w_down: torch.Tensor      # [E, hidden, inter]

    @classmethod
    def random(cls, experts: int, hidden: int, inter: int, gen: torch.Generator) -> "Experts":
        def normal(rows, cols):
            return torch.randn((experts, rows, cols), generator=gen, device="cuda") * cols ** -0.5
        e = cls(normal(2 * inter, hidden).bfloat16(), normal(hidden, inter).bfloat16())
        e.master = [e.w_gate_up.float(), e.w_down.float()]
        e.grads = [torch.zeros_like(m) for m in e.master]
        return e

    def step(self, lr: float) -> None:
        for w, m, g in zip((self.w_gate_up, self.w_down), self.master, self.grads):
            m.sub_(g, alpha=lr)
            w.copy_(m)
            g.zero_()


def forward(buf: ep.Buffer, experts: Experts, x, ids, scores, save: bool = False):
    """The layer's output for tokens x [T, hidden]; with save, what the backward pass needs."""
    d = buf.dispatch(x, scores, ids)
    if not save:
        return buf.combine(buf.expert_ffn(d.recv_x, experts.w_gate_up, experts.w_down), scores)
    y, h, gate_up = buf.expert_ffn(d.recv_x, experts.w_gate_up, experts.w_down, save=True)
    return buf.combine(y, scores), (d, y, h, gate_up)


def train_step(buf: ep.Buffer, experts: Experts, x, ids, scores, target):
    """Loss of the layer against target; adds the experts' gradients to experts.grads and
    returns (loss, gradient of x, gradient of scores)."""
    out, (d, y, h, gate_up) = forward(buf, experts, x, ids, scores, save=True)
    diff = out.float() - target.float()
    loss = diff.square().mean()
    grad_out = (diff * (2.0 / diff.numel())).bfloat16()
    grad_y, grad_scores = buf.combine_backward(grad_out, y, scores)
    grad_rows, _, _ = buf.expert_ffn_backward(grad_y, d.recv_x, experts.w_gate_up, experts.w_down,
                                              gate_up, h, grad_w_gate_up=experts.grads[0],
                                              grad_w_down=experts.grads[1], accumulate=True)
    grad_x, _ = buf.dispatch_backward(grad_rows, x.shape[0])
    return loss, grad_x, grad_scores


def quantise(w: torch.Tensor, group: int = 128) -> ep.W4:
    """4-bit codes of w [E, rows, cols]: per group of a row, 16 steps from its least to its
    greatest element, with the zero point on a step."""
    v = w.float().view(*w.shape[:2], -1, group)
    lo, hi = v.amin(-1).clamp(max=0.0), v.amax(-1).clamp(min=0.0)
    scale = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
    zero = (-lo / scale.float()).round().clamp(0, 15)
    q = (v / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8)
    q = q.view(*w.shape[:2], -1, 2)
    return ep.W4((q[..., 0] | (q[..., 1] << 4)).contiguous(), scale, zero.to(torch.uint8))


def decode_step(buf: ep.Buffer, w_gate_up: ep.W4, w_down: ep.W4, x, ids, scores):
    """The layer's output for a batch of single tokens, on 4-bit experts."""
    d = buf.dispatch(x, scores, ids)
    return buf.combine(buf.expert_ffn_w4(d.recv_x, w_gate_up, w_down), scores)


def quantise_fp4(w: torch.Tensor) -> ep.FP4:
    """w [E, rows, cols] as e2m1 with a scale for 16 elements and one for each expert."""
    return ep.quantize_fp4(w, "nv", w.abs().amax((1, 2)).float() / (6 * 448))


def main(tokens: int = 2048, hidden: int = 512, inter: int = 256, experts: int = 16, topk: int = 4,
         steps: int = 30, batch: int = 24, say=print) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    target, layer = (Experts.random(experts, hidden, inter, gen) for _ in range(2))
    buf = ep.Buffer(tokens, hidden, experts, 1, topk)
    x = torch.randn((tokens, hidden), generator=gen, device="cuda").bfloat16()
    ids, scores = ep.route(torch.randn((tokens, experts), generator=gen, device="cuda"), topk)
    want = forward(buf, target, x, ids, scores)
    losses = []
    for i in range(steps):
        loss, _, _ = train_step(buf, layer, x, ids, scores, want)
        layer.step(lr=200.0)
        losses.append(float(loss))
        if i % 10 == 0 or i == steps - 1:
            say(f"step {i:3d}: loss {losses[-1]:.5f}")
    out = forward(buf, layer, x[:batch], ids[:batch].contiguous(), scores[:batch].contiguous()).float()
    w4 = quantise(layer.w_gate_up), quantise(layer.w_down)
    got = decode_step(buf, *w4, x[:batch], ids[:batch].contiguous(), scores[:batch].contiguous())
    off = float((got.float() - out).norm() / out.norm())
    say(f"decoded {batch} tokens on 4-bit experts: {100 * off:.1f}% from the bf16 layer's output")
    got = buf.moe_layer(x[:batch], scores[:batch].contiguous(), ids[:batch].contiguous(),
                        quantise_fp4(layer.w_gate_up), quantise_fp4(layer.w_down))
    off_fp4 = float((got.float() - out).norm() / out.norm())
    say(f"and on experts in 4-bit floating point: {100 * off_fp4:.1f}%")
    assert buf.device_error() == 0
    buf.close()
    return {"losses": losses, "decode_off": off, "decode_fp4_off": off_fp4}


if __name__ == "__main__":
    main()
