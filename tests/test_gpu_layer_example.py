"""GPU test of the layer operators used together: the gradients of the example's
block against torch.autograd of the same block in float64, and its training."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import layer_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def rms(x, w):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * w


@pytest.mark.parametrize("tokens", [200, 37])
def test_block_gradients(tokens):
    """Each product's operands carry E4M3's rounding, 2^-4 of a value at most and
    about 2.6 % in the 2-norm; independent roundings add in squares.  The
    longest path to a gradient has six such operands behind it (and one product
    of two more), so its 2-norm is within 2.6 % sqrt(8) = 7.4 %; 15 % allows for
    twice that."""
    import fp8_layer as ex
    block = ex.Block(tokens, 256, 384, 130, p=0.2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(tokens, 256, device="cuda").normal_(generator=gen).to(torch.bfloat16)
    dout = torch.empty(tokens, 130, device="cuda").normal_(generator=gen).to(torch.bfloat16)
    out = block.forward(x, 5).clone()
    dx = block.backward(x, dout, 5)

    f = torch.from_numpy(ref.factors(tokens, 256, 0.2, seed=3, tensor_index=0, step=5)).cuda()
    xs = x.double().requires_grad_()
    layers = [block.up, block.down, block.head, block.norm1, block.norm2]
    up, down, head, g1, g2 = [m.weight.double().requires_grad_() for m in layers]
    # ReLU's mask from the block's own values, which rounding decides near zero
    a = (rms(xs, g1) @ up.T) * (block.a > 0)
    want = rms(xs + f * (a @ down.T), g2) @ head.T
    want.backward(dout.double())
    off = lambda got, exact: ((got.double() - exact).norm() / exact.norm()).item()  # noqa: E731
    assert off(out, want.detach()) <= 0.15
    assert off(dx, xs.grad) <= 0.15
    for m, w in zip(layers, (up, down, head, g1, g2)):
        assert off(m.grad, w.grad) <= 0.15


def test_training_lowers_the_loss():
    import fp8_layer as ex
    losses = ex.train(tokens=128, width=256, hidden=384, steps=60, lr=3e-3)
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
    assert losses == ex.train(tokens=128, width=256, hidden=384, steps=60, lr=3e-3), "two runs differ"
