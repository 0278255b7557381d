"""GPU test of the layer operators used together as a transformer block: its gradients
against torch.autograd of the same block in float64, and that it trains the same twice."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w


def turned(x, cos, sin):
    """Heads [tokens, heads, dim] turned by their token's angles, halves as pairs."""
    a, b = x.chunk(2, -1)
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("tokens,heads,kv_heads", [(200, 4, 2), (37, 2, 1)])
def test_block_gradients(tokens, heads, kv_heads):
    """Each 8-bit operand carries a rounding of 2^-4 of a value at most, about 2.6 % in the
    2-norm, and independent ones add in squares.  The longest way to a gradient (the inputs',
    through both halves) has sixteen operands behind it, counting those of the forward pass
    that its factors come from: 2.6 % sqrt(16) = 10.4 %; 21 % allows for twice that."""
    import fp8_transformer_block as ex
    width, hidden = 256, 392
    block = ex.Block(tokens, width, hidden, heads, kv_heads, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for m in (block.norm1, block.norm2, block.q_norm, block.k_norm):
        m.weight += 0.2 * torch.empty_like(m.weight).normal_(generator=gen)
    x = torch.empty(tokens, width, device="cuda").normal_(generator=gen).to(torch.bfloat16)
    dout = torch.empty(tokens, width, device="cuda").normal_(generator=gen).to(torch.bfloat16)
    out = block.forward(x).clone()
    dx = block.backward(x, dout)

    dim = width // heads
    xs = x.double().requires_grad_()
    q, k, v, o, gate, up, down, g1, g2, gq, gk = leaves = [m.weight.double().requires_grad_() for m in block.layers]
    n1 = rms(xs, g1)
    cos, sin = block.cos.double(), block.sin.double()
    qh = turned(rms((n1 @ q.T).view(tokens, heads, dim), gq), cos, sin).transpose(0, 1)
    kh = turned(rms((n1 @ k.T).view(tokens, kv_heads, dim), gk), cos, sin).transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    vh = (n1 @ v.T).view(tokens, kv_heads, dim).transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    scores = (qh @ kh.transpose(1, 2) * dim ** -0.5).masked_fill(torch.ones(tokens, tokens, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    h = xs + (torch.softmax(scores, -1) @ vh).transpose(0, 1).reshape(tokens, -1) @ o.T
    n2 = rms(h, g2)
    a = n2 @ gate.T
    want = h + (a * torch.sigmoid(a) * (n2 @ up.T)) @ down.T
    want.backward(dout.double())
    off = lambda got, exact: ((got.double() - exact).norm() / exact.norm()).item()  # noqa: E731
    assert off(out, want.detach()) <= 0.21
    assert off(dx, xs.grad) <= 0.21
    for m, w in zip(block.layers, leaves):
        assert off(m.grad, w.grad) <= 0.21


def test_training_runs_the_same_twice():
    import fp8_transformer_block as ex
    losses = ex.train(tokens=130, width=384, hidden=520, steps=6)
    assert np.isfinite(losses).all() and losses == ex.train(tokens=130, width=384, hidden=520, steps=6)
