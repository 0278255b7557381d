"""GPU tests of how near the gated activation and its gradients are to float64: of fp32
matrices by bounds that only fp32's own arithmetic meets, down to its subnormal numbers, and
of BF16 matrices at every finite value."""
import numpy as np
import pytest
import torch

import activation_reference as act
import precision_states_gb300 as ps
from test_gpu_layer import UNIT, blank, f64, matrix

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
KINDS = ["silu", "gelu_tanh", "gelu", "relu"]


def bounds(g, kind):
    """f, f', and bounds on either's absolute error in fp32, in units of 2^-24 (half a unit in
    the last place at most) of each part's value.

    silu: the exponential of -|g| is off by two units in the last place, 4 units; of s and 1 - s,
    one is r = 1 / (1 + e), off by 4 e / (1 + e) <= 2 and two roundings, and the other e r, off
    by 4 / (1 + e) <= 4 and three: 7.  f: one more, 8.  f' = s + (f (1 - s)) z': 7 of s, and of
    the second term 8 + 7 and a product, 16, and a rounding of the sum.
    gelu_tanh: z carries 6 roundings (its cubic term's factor three, the sum's, the last factor
    two), each worth |z| in the exponential: 6 |z| more in s, 1 - s and f; z' carries 6, and one
    more product.
    gelu: below 0, s is the fitted factor (8, with a reciprocal that is one off) times an
    exponential of two units in the last place (4), whose argument's rounding is put right (2) and
    a product: 15; above 0 it is 1 less that, which is no more, and a rounding: 16.  f: 17.  f' = s +
    g bell / sqrt(2 pi): 16 of s, of the second term the bell's 6, the factor's two, a product: 9,
    and a rounding of the sum.
    Subnormal numbers are kept: the exponential, s and their products are each off by at most a
    few 2^-149 more, 2^-146 (1 + |g|) and as much times z' in f'."""
    with np.errstate(all="ignore"):
        if kind == "relu":
            return np.maximum(g, 0.0), (g > 0).astype(np.float64), 0 * g, 0 * g
        tiny = 2.0 ** -146 * (1 + np.abs(g))
        if kind == "gelu":
            s, second = act.phi(g), g * np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
            return g * s, s + second, E24 * 17 * np.abs(g * s) + tiny, E24 * (16 * s + 9 * np.abs(second) + np.abs(s + second)) + tiny
        z, dz, more = g, np.ones_like(g), 0.0
        if kind == "gelu_tanh":
            c = 2 * np.sqrt(2 / np.pi)
            z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)
            more = 6 * np.abs(z)
        s, n = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
        f = g * s
        second = np.where(s * n == 0, 0.0, f * n * dz)
        # where the exponential underflows nothing is left of the terms that it carries
        return (f, s + second, E24 * np.where(f == 0, 0.0, (8 + more) * np.abs(f)) + tiny,
                E24 * (np.where(s == 0, 0.0, (7 + more) * s) + np.where(second == 0, 0.0, (16 + 2 * more + 7) * np.abs(second)) + np.abs(s + second))
                + tiny * (1 + dz))


def near(got, want, d, dtype="f32"):
    """Within d before one rounding to the type (half a step; 2^-150 or 2^-134 among its
    subnormal numbers)."""
    err, half = np.abs(f64(got) - want), 2.0 ** -150 if dtype == "f32" else 2.0 ** -134
    tol = UNIT[dtype] * (np.abs(want) + d) + d + half
    assert (err <= tol).all(), f"worst {np.max(err / tol)} of the bound, at {np.unravel_index(np.argmax(err / tol), err.shape)}"


def gates(rows, cols, pad=0):
    """From -16 to 16, and their sixteenths."""
    g = matrix(rows, cols, "f32", 1, pad)
    g.copy_(torch.linspace(-16, 16, rows * cols, device="cuda").view(rows, cols))
    g[1::2] /= 16
    return g


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("factor", [1.0, 1e10, 1e-20])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_forward(kind, factor, pad):
    """The factor: what up makes of an activation that is small, or subnormal."""
    rows, cols = 40, 1024
    g, u = gates(rows, cols, pad), matrix(rows, cols, "f32", 2, pad) * factor
    f, _, d, _ = bounds(f64(g), kind)
    y = blank(rows, cols, "f32", pad)
    ps.opt_gated(g, activation=kind, y=y)
    near(y, f, d)
    ps.opt_gated(g, u, activation=kind, y=y)
    near(y, f * f64(u), d * np.abs(f64(u)))


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_gradients(kind, turned, pad):
    rows, cols = 40, 1024
    g, u, dy = gates(rows, cols, pad), matrix(rows, cols, "f32", 2, pad), matrix(rows, cols, "f32", 3, pad) * 1e10
    f, df, d, dd = bounds(f64(g), kind)
    dg, du = blank(rows, cols, "f32", pad), blank(rows, cols, "f32", pad)
    t = ps.e4m3_storage(cols, rows)
    more = dict(y_codes_t=t) if turned else {}
    ps.opt_gated_backward(dy, g, u, activation=kind, dgate=dg, dup=du, **more)
    dv, uv = f64(dy), f64(u)
    # dy f' may round among the subnormal numbers before up multiplies it
    near(dg, dv * df * uv, (np.abs(dv) * dd + 2.0 ** -149 + 2 * E24 * np.abs(dv * df)) * np.abs(uv))
    near(du, dv * f, np.abs(dv) * d)


def test_fp32_gelu_far_below():
    """Where s is below 2^-126 an up of 1e10 still has its part of it."""
    g, u = torch.full((1, 8), -13.25, device="cuda"), torch.full((1, 8), 1e10, device="cuda")
    y, dg = blank(1, 8, "f32"), blank(1, 8, "f32")
    ps.opt_gated(g, u, activation="gelu", y=y)
    ps.opt_gated_backward(u, g, activation="gelu", dgate=dg)
    f, df, _, _ = bounds(np.float64(-13.25), "gelu")
    assert abs(y[0, 0].item() / (f * 1e10) - 1) < 1e-3 and abs(dg[0, 0].item() / (df * 1e10) - 1) < 1e-3


@pytest.mark.parametrize("kind", KINDS)
def test_bf16_at_every_finite_value(kind):
    """By the bound of BF16's fast forms, whose s is 0 below 2^-126."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda")
    bits = bits[(bits & 0x7F80) != 0x7F80].to(torch.int16).view(255, 256)
    g = bits.view(torch.bfloat16)
    y, dg = blank(255, 256, "bf16"), blank(255, 256, "bf16")
    ps.opt_gated(g, activation=kind, y=y)
    ps.opt_gated_backward(torch.ones_like(g), g, activation=kind, dgate=dg)
    f, df, d, dd = act.activation(f64(g), kind)
    near(y, f, d, "bf16")
    near(dg, df, dd, "bf16")
