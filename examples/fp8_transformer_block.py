"""A transformer block trained with 8-bit products and with its activations kept in 8
bits, from its inputs to the parameter step, on one GPU:

    python examples/fp8_transformer_block.py [--tokens N] [--width D] [--hidden F] [--steps S]

Forward: the norm in E4M3 codes; query, key and value products; the norm of each
head with the position rotation, its inputs kept in 8 bits; attention (torch, the
only thing that is not this library's); the output product; the residual norm; gate
and up products; the gated activation, which writes the down product's operand and
keeps both of its inputs in 8 bits.  Backward: the gated activation's gradients come
from the kept inputs as the operands of the next products in both orientations, the
heads' from the kept heads, and each weight gradient's other operand is the forward
pass's own codes turned.  What is held from one pass to the other in more than 8 bits
is the residual stream, one number per row, and what attention wants.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_states_gb300 as ps  # noqa: E402

BF16 = torch.bfloat16


class Linear:
    """y = x W^T with all three products on E4M3 operands; W and its gradient are fp32."""

    def __init__(self, n_out, n_in, gen):
        self.weight = torch.empty(n_out, n_in, device="cuda").normal_(0.0, n_in ** -0.5, generator=gen)
        self.grad = torch.zeros_like(self.weight)
        self.w, self.wt = ps.e4m3_storage(n_out, n_in), ps.e4m3_storage(n_in, n_out)
        self.refresh()

    def refresh(self):
        """The weight's codes in both orientations, after each step."""
        ps.opt_quantize(self.weight, *self.w, *self.wt, block_rows=128)

    def forward(self, x, out):
        ps.opt_matmul(*x, *self.w, out)

    def backward(self, dy, dy_t, x_t, dx, add=False):
        """dx (+)= dy W and grad = dy^T x, from operands."""
        ps.opt_matmul(*dy, *self.wt, dx, addend=dx if add else None)
        ps.opt_matmul(*dy_t, *x_t, self.grad)


class Gain:
    """A norm's weight and its gradient."""

    def __init__(self, width):
        self.weight, self.grad = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")


def rotation(positions, dim, base=1e4):
    """The rotation's tables, float32, from angles in float64."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64) / dim)
    return torch.cos(angle).float().cuda(), torch.sin(angle).float().cuda()


def attention(q, k, v, heads, kv_heads, dim):
    """Causal attention of one sequence; groups of query heads share a key head."""
    t = q.shape[0]
    q, k, v = (x.float().view(t, -1, dim).transpose(0, 1) for x in (q, k, v))
    k, v = (x.repeat_interleave(heads // kv_heads, 0) for x in (k, v))
    scores = q @ k.transpose(1, 2) * dim ** -0.5
    scores = scores.masked_fill(torch.ones(t, t, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    return (torch.softmax(scores, -1) @ v).transpose(0, 1).reshape(t, -1)


class Block:
    """h = x + o(attention(q, k, v)); out = h + down(silu(gate(norm(h))) up(norm(h)))."""

    def __init__(self, tokens=512, width=768, hidden=2304, heads=12, kv_heads=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.heads, self.kv_heads, self.dim = tokens, heads, kv_heads, width // heads
        kv = kv_heads * self.dim
        self.q, self.k, self.v = Linear(width, width, gen), Linear(kv, width, gen), Linear(kv, width, gen)
        self.o = Linear(width, width, gen)
        self.gate, self.up, self.down = Linear(hidden, width, gen), Linear(hidden, width, gen), Linear(width, hidden, gen)
        self.norm1, self.norm2, self.q_norm, self.k_norm = Gain(width), Gain(width), Gain(self.dim), Gain(self.dim)
        self.cos, self.sin = rotation(tokens, self.dim)
        new = lambda n: torch.empty(tokens, n, dtype=BF16, device="cuda")  # noqa: E731
        held = lambda n: ps.e4m3_storage(tokens, n)  # noqa: E731
        turned = lambda n: ps.e4m3_storage(n, tokens)  # noqa: E731
        # kept from the forward to the backward pass
        self.n1, self.n2, self.q_kept, self.k_kept, self.o_in = held(width), held(width), held(width), held(kv), held(width)
        self.gate_kept, self.up_kept = held(hidden), held(hidden)
        self.rstd1, self.rstd2 = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.h, self.out = new(width), new(width)
        # scratch of either pass
        self.w1, self.w2, self.kv1, self.kv2, self.kv3, self.f1, self.f2 = new(width), new(width), new(kv), new(kv), new(kv), new(hidden), new(hidden)
        self.act = held(hidden)
        self.d_w, self.d_kv, self.t_w, self.t_kv, self.x_t = held(width), held(kv), turned(width), turned(kv), turned(width)
        self.d_gate, self.d_up = held(hidden), held(hidden)
        self.t_gate, self.t_up, self.act_t = turned(hidden), turned(hidden), turned(hidden)
        self.dn, self.dh, self.dx = new(width), new(width), new(width)
        self.layers = [self.q, self.k, self.v, self.o, self.gate, self.up, self.down, self.norm1, self.norm2, self.q_norm, self.k_norm]
        params, grads = [m.weight.view(-1) for m in self.layers], [m.grad.view(-1) for m in self.layers]
        self.plan = ps.Plan(params, grads, [torch.zeros_like(t) for t in params], [torch.zeros_like(t) for t in params])

    def _turn(self):
        return dict(cos=self.cos, sin=self.sin)

    def forward(self, x):
        ps.opt_rms_norm(x, self.norm1.weight, rstd=self.rstd1, codes=self.n1[0], scales=self.n1[1])
        q, k, v = self.w1, self.kv1, self.kv3
        for layer, out in ((self.q, q), (self.k, k), (self.v, v)):
            layer.forward(self.n1, out)
        ps.opt_head_norm(q, self.q_norm.weight, self.w2, k, self.k_norm.weight, self.kv2, q_kept=self.q_kept, k_kept=self.k_kept, **self._turn())
        self.leaves = [t.detach().clone().requires_grad_() for t in (self.w2, self.kv2, v)]
        self.o_out = attention(*self.leaves, self.heads, self.kv_heads, self.dim).to(BF16)
        ps.opt_quantize(self.o_out.detach(), *self.o_in)
        self.o.forward(self.o_in, self.w1)
        ps.opt_rms_norm(self.w1, self.norm2.weight, rstd=self.rstd2, residual=x, h=self.h, codes=self.n2[0], scales=self.n2[1])
        self.gate.forward(self.n2, self.f1)
        self.up.forward(self.n2, self.f2)
        ps.opt_gated(self.f1, self.f2, codes=self.act[0], scales=self.act[1], gate_kept=self.gate_kept, up_kept=self.up_kept)
        self.down.forward(self.act, self.w1)
        ps.opt_dropout(self.w1, self.out, 0.0, residual=self.h)
        return self.out

    def backward(self, x, dout):
        # the gated half
        ps.opt_quantize(dout, *self.d_w, *self.t_w)
        ps.opt_matmul(*self.d_w, *self.down.wt, self.f1)
        ps.opt_gated_backward(self.f1, self.gate_kept, self.up_kept, dgate_codes=self.d_gate, dgate_codes_t=self.t_gate,
                              dup_codes=self.d_up, dup_codes_t=self.t_up, y_codes_t=self.act_t)
        ps.opt_matmul(*self.t_w, *self.act_t, self.down.grad)
        ps.opt_dequantize(*self.n2, codes_t=self.x_t[0], scales_t=self.x_t[1])
        self.gate.backward(self.d_gate, self.t_gate, self.x_t, self.dn)
        self.up.backward(self.d_up, self.t_up, self.x_t, self.dn, add=True)
        ps.opt_rms_norm_backward(self.dn, self.h, self.norm2.weight, self.rstd2, self.dh, dh_in=dout, dweight=self.norm2.grad)
        # attention
        ps.opt_quantize(self.dh, *self.d_w, *self.t_w)
        ps.opt_dequantize(*self.o_in, codes_t=self.x_t[0], scales_t=self.x_t[1])
        self.o.backward(self.d_w, self.t_w, self.x_t, self.dn)
        dq_out, dk_out, dv = (g.to(BF16) for g in torch.autograd.grad(self.o_out, self.leaves, self.dn))
        ps.opt_head_norm_backward(dq_out, self.q_kept, self.q_norm.weight, self.w1, dk_out, self.k_kept, self.k_norm.weight, self.kv1,
                                  dq_weight=self.q_norm.grad, dk_weight=self.k_norm.grad, **self._turn())
        ps.opt_dequantize(*self.n1, codes_t=self.x_t[0], scales_t=self.x_t[1])
        for i, (layer, dy, d, t) in enumerate(((self.q, self.w1, self.d_w, self.t_w), (self.k, self.kv1, self.d_kv, self.t_kv),
                                               (self.v, dv, self.d_kv, self.t_kv))):
            ps.opt_quantize(dy, *d, *t)
            layer.backward(d, t, self.x_t, self.dn, add=i > 0)
        ps.opt_rms_norm_backward(self.dn, x, self.norm1.weight, self.rstd1, self.dx, dh_in=self.dh, dweight=self.norm1.grad)
        return self.dx

    def update(self, step, lr=1e-3, max_norm=1.0):
        self.plan.grad_norm(max_norm, sync=False)
        self.plan.adamw_step(ps.hparams(lr=lr, weight_decay=0.01), step, self.plan.norm_buffer())
        for m in self.layers[:7]:
            m.refresh()


def train(tokens=512, width=768, hidden=2304, steps=50, lr=1e-3, seed=0):
    """Losses of `steps` steps on one fixed batch and random target."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.empty(tokens, width, device="cuda").normal_(generator=gen).to(BF16)
    target = torch.empty(tokens, width, device="cuda").normal_(generator=gen)
    block = Block(tokens, width, hidden, seed=seed)
    losses = []
    for step in range(1, steps + 1):
        diff = block.forward(x).float() - target
        losses.append(diff.square().mean())
        block.backward(x, (diff * (2.0 / diff.numel())).to(BF16))
        block.update(step, lr)
    assert ps.opt_layer_status() == 0
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 512), ("width", 768), ("hidden", 2304), ("steps", 50)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    losses = train(a.tokens, a.width, a.hidden, a.steps)
    print("loss: first %.4f, last %.4f over %d steps" % (losses[0], losses[-1], len(losses)))
