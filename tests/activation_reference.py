"""Definitions in float64 of the operators between a block's products (the gated
activation, the heads' norm with rotation) and bounds on what fp32 arithmetic may
miss them by.  Test infrastructure only."""
import numpy as np
import torch

import layer_reference as ref

E24 = 2.0 ** -24
UNIT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 2.0 ** -126                # below it fp32 has fewer bits


def phi(x):
    """The normal distribution function by the complement of erf (1 + erf has no digits left
    below -8)."""
    return 0.5 * torch.special.erfc(torch.from_numpy(np.asarray(x)) * -np.sqrt(0.5)).numpy()


def activation(g, kind):
    """f, f', and bounds on the absolute error of either in fp32.

    silu, gelu_tanh: z in at most four roundings; exp(-|z|) is off by |z| times the
    error of its argument (5 roundings with the factor log2 e) and 4 units of 2^-24 of
    its own, and s and 1 - s by 4 more (sum, reciprocal, product); f by one more.  f' is
    s + f (1 - s) z', with five more roundings in the second term; 1 - s may be formed as
    that, off by 2^-24.  s is 0 where it would be below 2^-126 in BF16,
    which leaves f off by |g| 2^-126 and f' by 2^-126 (1 + |g| z').  gelu: the
    distribution function below 0 is an exponential (4 units, and g^2 for the rounding of its
    argument, half of g^2 formed with two) times a fitted factor (8), with three products; above
    0 it is 1 less that."""
    with np.errstate(all="ignore"):
        if kind == "relu":
            f, df = np.maximum(g, 0.0), (g > 0).astype(np.float64)
            return f, df, 0 * f, 0 * f
        if kind == "gelu":
            s, bell = phi(g), g * np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
            far, off = TINY * (1 + np.abs(g)), 17 + np.minimum(g * g, 300)
            return (g * s, s + bell, E24 * off * np.abs(g * s) + far,
                    far + E24 * (off * s + (np.minimum(g * g, 300) + 10) * np.abs(bell) + np.abs(s + bell)))
        z, dz = g, np.ones_like(g)
        if kind == "gelu_tanh":
            c = 2 * np.sqrt(2 / np.pi)
            z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)
        s, n = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
        f, second = g * s, g * s * n * dz
        second = np.where(s * n == 0, 0.0, second)
        off = np.minimum(5 * np.abs(z), 600) + 10
        far, far_slope = TINY * (1 + np.abs(g)), TINY * (1 + np.abs(g * dz))
        return (f, s + second, E24 * off * np.abs(f) + far,
                E24 * (off * s + np.minimum(np.abs(f * dz), 600) + (2 * off + 6) * np.abs(second) + np.abs(s + second)) + far_slope)


def check_codes(codes, scales, want, d):
    """Codes and scales of values that are within d of `want`: the scale is the rule's
    for a value between, and each code within half a step of its value."""
    rows, cols = want.shape
    e = ref.scale_bytes_of(scales, rows, cols) - 127
    size = np.abs(want)
    lo, hi = ref.block_exponents(size - np.minimum(d, size), 1), ref.block_exponents(size + d, 1)
    assert ((e >= lo) & (e <= hi)).all()
    step = 2.0 ** np.repeat(e, 128, 1)[:, :cols].astype(np.float64)
    v = ref.values(codes, scales)
    assert (np.abs(v - want) <= np.maximum(size * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * d).all()


def check_kept(codes, scales, x):
    """Codes and scales of x (float32 values) exactly as the quantizer makes them."""
    rows, cols = x.shape
    e = ref.block_exponents(x.astype(np.float64), 1)
    assert (ref.scale_bytes_of(scales, rows, cols) - 127 == e).all()
    got, want = codes.cpu().numpy(), ref.encode(x, e)
    assert (got[np.isfinite(x)] == want[np.isfinite(x)]).all() and (got & 0x7F == want & 0x7F).all()


def untouched(scales, rows, cols, fill):
    """Scale bytes of rows and blocks that do not exist still hold `fill`."""
    unused = np.ones(scales.numel(), bool)
    unused[ref.tile_places(rows, -(-cols // 128)).reshape(-1)] = False
    return (scales.cpu().numpy()[unused] == fill).all()


def turn(n, cos, sin, rot, interleaved, back=False):
    """Heads [rows, heads, dim] turned by cos and sin [rows, rot / 2] (or back), and the
    sum of its terms' magnitudes."""
    out, size = n.copy(), np.abs(n)
    if rot == 0:
        return out, size
    c, s = cos[:, None, :], (-sin if back else sin)[:, None, :]
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = n[..., i], n[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i], size[..., j] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, size


def head_norm(x, w, eps, cos, sin, rot, interleaved):
    """Outputs of heads x [rows, heads, dim] and a bound on their error: the sum of squares
    (dim / 32 + 14 roundings, halved by the root), the root (4), the products (5)."""
    dim = x.shape[-1]
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        y, size = turn(x * rstd * w, cos, sin, rot, interleaved)
    return y, E24 * (dim / 64 + 16) * size


def head_norm_backward(dout, x, w, eps, cos, sin, rot, interleaved):
    """dx and its bound, the weight's gradient and the sum of its terms' magnitudes."""
    dim = x.shape[-1]
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g, size = turn(dout, cos, sin, rot, interleaved, back=True)
    t = g * w
    dx = rstd * (t - x * rstd ** 2 * (t * x).mean(-1, keepdims=True))
    first = rstd * size * np.abs(w)
    second = np.abs(x) * rstd ** 3 * (size * np.abs(w * x)).mean(-1, keepdims=True)
    n = dim / 32 + 14
    d = E24 * ((n / 2 + 10) * first + (3 * n + 20) * second)
    terms = g * x * rstd
    return dx, d, terms.sum((0, 1)), (size * np.abs(x) * rstd).sum((0, 1))
