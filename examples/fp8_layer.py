"""A residual feed-forward block trained with 8-bit products, from its inputs to
the parameter step, on one GPU:

    python examples/fp8_layer.py [--tokens N] [--width D] [--hidden F] [--steps S]

Per step: the residual norm writes the block's input as BF16 and as E4M3 codes
with block scales; two products (the weights' codes are laid out once per step);
branch dropout and the second norm in one call; a product with the output
weight; then the same backward -- each gradient to codes in both orientations,
two products per weight, the norms' gradients -- and at the end the gradient
norm and one AdamW step over all parameters.  The loss is the mean squared
difference to a fixed random target.  No tensor library computes a product:
torch holds memory and does the loss and the ReLU.
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

    def __init__(self, n_out, n_in, tokens, gen):
        self.weight = torch.empty(n_out, n_in, device="cuda").normal_(0.0, n_in ** -0.5, generator=gen)
        self.grad = torch.zeros_like(self.weight)
        self.w, self.wt = ps.e4m3_storage(n_out, n_in), ps.e4m3_storage(n_in, n_out)
        self.dy, self.dyt = ps.e4m3_storage(tokens, n_out), ps.e4m3_storage(n_out, tokens)
        self.xt = ps.e4m3_storage(n_in, tokens)
        self.refresh()

    def refresh(self):
        """The weight's codes in both orientations, after each step."""
        ps.opt_quantize(self.weight, *self.w, *self.wt, block_rows=128)

    def forward(self, x_codes, out):
        ps.opt_matmul(*x_codes, *self.w, out)

    def backward(self, dy, x, dx):
        """dx = dy W and grad = dy^T x, from BF16 dy and x."""
        ps.opt_quantize(dy, *self.dy, *self.dyt)
        ps.opt_quantize(x, codes_t=self.xt[0], scales_t=self.xt[1])
        ps.opt_matmul(*self.dy, *self.wt, dx)
        ps.opt_matmul(*self.dyt, *self.xt, self.grad)


class Norm:
    """The gain of one residual norm, and what its backward pass needs."""

    def __init__(self, width, tokens):
        self.weight = torch.ones(width, device="cuda")
        self.grad = torch.zeros_like(self.weight)
        self.rstd = torch.empty(tokens, device="cuda")
        self.y = torch.empty(tokens, width, dtype=BF16, device="cuda")
        self.codes = ps.e4m3_storage(tokens, width)
        self.workspace = torch.empty(max(ps.opt_rms_norm_backward_workspace(tokens, width), 1), dtype=torch.uint8,
                                     device="cuda")


class Block:
    """out = head(norm2(x + dropout(down(relu(up(norm1(x)))))))."""

    def __init__(self, tokens=512, width=768, hidden=2304, n_out=768, p=0.1, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.p, self.seed, self.tokens = p, seed, tokens
        self.up, self.down = Linear(hidden, width, tokens, gen), Linear(width, hidden, tokens, gen)
        self.head = Linear(n_out, width, tokens, gen)
        self.norm1, self.norm2 = Norm(width, tokens), Norm(width, tokens)
        new = lambda n: torch.empty(tokens, n, dtype=BF16, device="cuda")  # noqa: E731
        self.a, self.branch, self.h, self.out = new(hidden), new(width), new(width), new(n_out)
        self.a_codes = ps.e4m3_storage(tokens, hidden)
        self.dn2, self.dh, self.dbranch, self.da, self.dn1, self.dx = new(width), new(width), new(width), new(hidden), new(width), new(width)
        layers = [self.up, self.down, self.head, self.norm1, self.norm2]
        params, grads = [m.weight.view(-1) for m in layers], [m.grad.view(-1) for m in layers]
        self.plan = ps.Plan(params, grads, [torch.zeros_like(t) for t in params], [torch.zeros_like(t) for t in params])

    def _draws(self, step):
        return dict(p=self.p, seed=self.seed, tensor_index=0, step=step)

    def forward(self, x, step):
        n1, n2 = self.norm1, self.norm2
        ps.opt_rms_norm(x, n1.weight, y=n1.y, rstd=n1.rstd, codes=n1.codes[0], scales=n1.codes[1])
        self.up.forward(n1.codes, self.a)
        self.a.relu_()
        ps.opt_quantize(self.a, *self.a_codes)
        self.down.forward(self.a_codes, self.branch)
        ps.opt_rms_norm(self.branch, n2.weight, y=n2.y, rstd=n2.rstd, residual=x, h=self.h, codes=n2.codes[0],
                        scales=n2.codes[1], **self._draws(step))
        self.head.forward(n2.codes, self.out)
        return self.out

    def backward(self, x, dout, step):
        n1, n2 = self.norm1, self.norm2
        self.head.backward(dout, n2.y, self.dn2)
        ps.opt_rms_norm_backward(self.dn2, self.h, n2.weight, n2.rstd, self.dh, dx=self.dbranch, dweight=n2.grad,
                                 workspace=n2.workspace, **self._draws(step))
        self.down.backward(self.dbranch, self.a, self.da)
        self.da.mul_(self.a > 0)
        self.up.backward(self.da, n1.y, self.dn1)
        ps.opt_rms_norm_backward(self.dn1, x, n1.weight, n1.rstd, self.dx, dh_in=self.dh, dweight=n1.grad,
                                 workspace=n1.workspace)
        return self.dx

    def update(self, step, lr=1e-3, max_norm=1.0):
        self.plan.grad_norm(max_norm, sync=False)
        self.plan.adamw_step(ps.hparams(lr=lr, weight_decay=0.01), step, self.plan.norm_buffer())
        for m in (self.up, self.down, self.head):
            m.refresh()


def train(tokens=512, width=768, hidden=2304, steps=50, lr=1e-3, seed=0):
    """Losses of `steps` steps on one fixed batch."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.empty(tokens, width, device="cuda").normal_(generator=gen).to(BF16)
    target = torch.empty(tokens, width, device="cuda").normal_(generator=gen)
    block = Block(tokens, width, hidden, width, seed=seed)
    losses = []
    for step in range(1, steps + 1):
        diff = block.forward(x, step).float() - target
        losses.append(diff.square().mean())
        block.backward(x, (diff * (2.0 / diff.numel())).to(BF16), step)
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
