"""GPU tests of the training-layer operators against their definitions in
float64 (tests/layer_reference.py), at the sizes, layouts and values where they
can go wrong, and of their gradients against differences.

Tolerances.  An output of a type with unit roundoff u (2^-p for p
significant bits: 2^-8 BF16, 2^-24 fp32),
formed in fp32 with an absolute error of at most d and rounded once, is within
u |y| + 2 d of the exact y.  d is stated at each test from the number of fp32
roundings (each 2^-24 relative) of the terms that form the output.  E4M3 codes
of exactly known inputs are compared for equality; codes of computed values lie
within half of the grid's spacing, 2^-4 of the value or 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import precision_states_gb300 as ps

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E24 = 2.0 ** -24
DRAW = dict(seed=0x1234567890ABCDEF, tensor_index=5, step=77)


def matrix(rows, cols, dtype, seed, pad=0, shift=0, std=1.0):
    """A rows x cols tensor whose rows are `pad` elements longer, `shift`
    elements into its allocation."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.empty(rows * (cols + pad) + shift, device="cuda").normal_(0.0, std, generator=g).to(TD[dtype])
    return flat[shift:].view(rows, cols + pad)[:, :cols]


def blank(rows, cols, dtype, pad=0):
    return torch.full((rows, cols + pad), 7.0, dtype=TD[dtype], device="cuda")[:, :cols]


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, dtype, d):
    err = np.abs(f64(got) - want)
    tol = UNIT[dtype] * np.abs(want) + 2 * d
    assert (err <= tol).all(), f"worst {np.max(err - tol)} over, at {np.unravel_index(np.argmax(err - tol), err.shape)}"


# ------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift,residual,p", [
    (1, 1, 0, 0, False, 0.5), (1, 7, 0, 0, True, 0.1), (1, 4096, 0, 0, True, 0.1), (3, 8, 8, 0, True, 0.3),
    (5, 13, 0, 0, False, 0.25), (33, 257, 3, 1, True, 0.1), (64, 768, 0, 0, False, 0.0), (40, 512, 64, 0, True, 0.9),
    (17, 100, 0, 0, True, 1.0), (70001, 1, 2, 0, False, 0.4)])
def test_dropout(dtype, rows, cols, pad, shift, residual, p):
    x = matrix(rows, cols, dtype, 1, pad, shift)
    r = matrix(rows, cols, dtype, 2) if residual else None
    y = blank(rows, cols, dtype, pad)
    ps.opt_dropout(x, y, p, residual=r, **DRAW)
    f = ref.factors(rows, cols, p, **DRAW)
    scaled = f64(x) * f
    want = scaled + (f64(r) if residual else 0.0)
    within(y, want, dtype, E24 * (2 * np.abs(scaled) + np.abs(want)))     # factor, product, sum
    if not residual:
        assert ((f64(y) == 0) == ((f == 0) | (f64(x) == 0))).all()
    if pad:
        assert (y.as_strided((rows, pad), (cols + pad, 1), cols) == 7).all(), "wrote between the rows"


def test_dropout_layout_does_not_change_the_mask_and_aliasing():
    x = matrix(37, 136, "bf16", 3)
    y = torch.empty_like(x)
    ps.opt_dropout(x, y, 0.3, **DRAW)
    wide = torch.zeros(37, 139, dtype=torch.bfloat16, device="cuda")
    wide[:, :136] = x
    out = wide[:, :136]
    ps.opt_dropout(out, out, 0.3, **DRAW)                     # in place, unaligned rows
    assert torch.equal(out, y)
    again = x.view(-1)                                        # the same element numbers as one row
    z = torch.empty_like(again)
    ps.opt_dropout(again, z, 0.3, **DRAW)
    assert torch.equal(z.view(37, 136), y)
    ps.opt_dropout(x, z.view(37, 136), 0.3, **{**DRAW, "step": 78})
    assert not torch.equal(z.view(37, 136), y)


def test_dropout_rate_and_elements_past_2_32():
    """The kept fraction of 2^26 elements within 6 standard deviations; the
    element number of a late element of a tall matrix is 64 bits wide."""
    n = 1 << 26
    y = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    ps.opt_dropout(torch.ones_like(y), y, 0.1, **DRAW)
    t = round(65536 * 0.1)
    kept = (y != 0).sum().item() / n
    assert abs(kept - (1 - t / 65536)) <= 6 * (0.1 * 0.9 / n) ** 0.5
    rows, cols = (1 << 21) + 3, 4096                          # over 2^33 elements
    big = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    ps.opt_dropout(big, big, 0.5, **DRAW)
    import oracle
    for r, c in ((rows - 1, 4088), (1 << 20, 0), ((1 << 20) - 1, 4088)):
        g = (r * cols + c) // 8
        w = oracle.philox4x32_10([g & 0xFFFFFFFF, (g >> 32) | 0x80000000, DRAW["tensor_index"], DRAW["step"]],
                                 [DRAW["seed"] & 0xFFFFFFFF, DRAW["seed"] >> 32])
        want = [2.0 if ((w[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= 32768 else 0.0 for j in range(8)]
        assert big[r, c:c + 8].tolist() == want


# ------------------------------------------------------------------ rms norm
def norm_reference(x, res, w, p, eps):
    f = ref.factors(*x.shape, p, **DRAW)
    scaled = f64(x) * f
    h = scaled + (f64(res) if res is not None else 0.0)
    dh = E24 * (2 * np.abs(scaled) + np.abs(h))
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, dh, rstd, h * rstd[:, None] * f64(w)


NORM_SHAPES = [(1, 1, 0), (1, 4096, 0), (3, 8, 0), (2, 127, 0), (5, 129, 3), (67, 768, 0), (130, 769, 0), (9, 2304, 8),
               (4, 5000, 0), (3, 16384, 0), (2, 33000, 0), (2, 40001, 1), (700, 136, 0), (512, 2048, 0), (513, 64, 0), (33, 32001, 0)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", NORM_SHAPES)
def test_rms_norm(dtype, wdtype, rows, cols, pad):
    full = (rows + cols) % 2 == 1
    p = 0.2 if full and rows * cols < 300000 else 0.0
    x = matrix(rows, cols, dtype, 4, pad)
    res = matrix(rows, cols, dtype, 5, std=3.0) if full else None
    w = (1 + 0.2 * matrix(1, cols, "f32", 6)[0]).to(TD[wdtype])
    h, y = blank(rows, cols, dtype), blank(rows, cols, dtype, pad)
    rstd = torch.empty(rows, device="cuda")
    codes, scales = ps.e4m3_storage(rows, cols)
    scales.fill_(0xEE)
    ps.opt_rms_norm(x, w, 1e-5, y=y, rstd=rstd, residual=res, h=h, codes=codes, scales=scales, p=p, **DRAW)
    hx, dh, sx, yx = norm_reference(x, res, w, p, 1e-5)
    within(h, hx, dtype, dh)
    # sum of squares: cols / 8 / threads sequential adds per thread and 10 levels, all positive
    deep = cols / 2048 * 8 + 20
    ds = sx * E24 * (deep + 6) + sx * E24 * 4
    assert (np.abs(f64(rstd) - sx) <= ds + sx * E24).all()
    dy = np.abs(yx) * (E24 * 3 + (ds / sx)[:, None]) + dh * sx[:, None] * np.abs(f64(w))
    within(y, yx, dtype, dy)
    # scales: exact except where the block's largest value is within its error of a boundary
    e = ref.scale_bytes_of(scales, rows, cols) - 127
    lo, hi = ref.block_exponents(np.abs(yx) - np.minimum(dy, np.abs(yx)), 1), ref.block_exponents(np.abs(yx) + dy, 1)
    assert ((e >= lo) & (e <= hi)).all()
    step = 2.0 ** np.repeat(e, 128, 1)[:, :cols].astype(np.float64)
    v = ref.values(codes, scales)
    assert (np.abs(v - yx) <= np.maximum(np.abs(yx) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * dy).all()
    unused = np.ones(scales.numel(), bool)
    unused[ref.tile_places(rows, -(-cols // 128)).reshape(-1)] = False
    assert (scales.cpu().numpy()[unused] == 0xEE).all(), "wrote scale bytes of rows or blocks that do not exist"


def test_rms_norm_codes_are_those_of_the_quantizer():
    """fp32 y and its codes come from the same values."""
    x = matrix(45, 900, "f32", 8)
    w = matrix(1, 900, "f32", 9)[0].contiguous()
    y = torch.empty_like(x)
    c1, s1 = ps.e4m3_storage(45, 900)
    c2, s2 = ps.e4m3_storage(45, 900)
    ps.opt_rms_norm(x, w, y=y, codes=c1, scales=s1)
    ps.opt_quantize(y, c2, s2)
    assert torch.equal(c1, c2) and torch.equal(s1, s2)


@pytest.mark.parametrize("cols", [4096, 769])
def test_rms_norm_special_rows(cols):
    x = matrix(6, cols, "f32", 10)
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e25                                        # squares overflow fp32
    x[5] = 1e-30                                       # squares vanish below eps
    w = torch.ones(cols, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    codes, scales = ps.e4m3_storage(6, cols)
    ps.opt_rms_norm(x, w, 1e-6, y=y, rstd=rstd, codes=codes, scales=scales)
    assert torch.isfinite(y[0]).all() and (y[1] == 0).all() and (codes[1] & 0x7F == 0).all()
    assert torch.isnan(y[2]).all() and (codes[2] == 0x7F).all()
    assert rstd[3] == 0 and torch.isnan(y[3, 7]) and (y[3, 8:] == 0).all() and codes[3, 7] == 0x7F
    assert (y[4] == 0).all() and torch.allclose(y[5], x[5] * 1e3, rtol=1e-6, atol=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(6000, 261), (1500, 260), (2000, 2047), (1300, 4101), (400, 8201), (400, 12301), (400, 8200)])
def test_rms_norm_drops_what_dropout_drops(dtype, rows, cols):
    """Many rows per CTA, rows that begin anywhere among the generator's calls."""
    x = matrix(rows, cols, dtype, 14)
    w = torch.ones(cols, device="cuda")
    want, h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    ps.opt_dropout(x, want, 0.3, **DRAW)
    ps.opt_rms_norm(x, w, 1e-5, y=y, rstd=rstd, h=h, p=0.3, **DRAW)
    assert torch.equal(h, want)
    dh_in, dh, dx = torch.full_like(x, 64.0), torch.empty_like(x), torch.empty_like(x)
    ps.opt_rms_norm_backward(x, h, w, rstd, dh, dh_in=dh_in, dx=dx, p=0.3, **DRAW)
    ps.opt_dropout(torch.ones_like(x), want, 0.3, **DRAW)
    assert (dh > 0).all() and torch.equal(dx != 0, want != 0)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", NORM_SHAPES)
def test_rms_norm_backward(dtype, wdtype, rows, cols, pad):
    full = (rows + cols) % 2 == 1
    p = 0.2 if full and rows * cols < 300000 else 0.0
    h = matrix(rows, cols, dtype, 11, pad)
    dy = matrix(rows, cols, dtype, 12)
    w = (1 + 0.2 * matrix(1, cols, "f32", 6)[0]).to(TD[wdtype])
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    dh_in = matrix(rows, cols, dtype, 13) if full else None
    dh, dx = blank(rows, cols, dtype), blank(rows, cols, dtype, pad) if p > 0 else None
    dw = torch.empty(cols, device="cuda")
    ps.opt_rms_norm_backward(dy, h, w, rstd, dh, dh_in=dh_in, dx=dx, dweight=dw, p=p, **DRAW)
    g, hh, s = f64(dy) * f64(w), f64(h), f64(rstd)[:, None]
    want = s * (g - hh * s * s * (g * hh).mean(1, keepdims=True))
    # mean(g h): cols / 2048 * 8 + 20 sequential roundings of terms |g h|; then five roundings of each term
    second = np.abs(s * hh * s * s) * np.abs(g * hh).mean(1, keepdims=True)
    d = E24 * (6 * np.abs(s * g) + (cols / 2048 * 8 + 30) * second)
    if full:
        want = want + f64(dh_in)
        d = d + E24 * np.abs(want)
    within(dh, want, dtype, d)
    if p > 0:
        f = ref.factors(rows, cols, p, **DRAW)
        within(dx, want * f, dtype, (d + 2 * E24 * np.abs(want)) * f)
    terms = f64(dy) * hh * s
    # at most ceil(rows / 1024) + 1024 sequential adds
    assert (np.abs(f64(dw) - terms.sum(0)) <= E24 * (min(rows, 1100) + 4) * np.abs(terms).sum(0)).all()


def test_rms_norm_backward_against_differences():
    """The gradient of sum(c y) + sum(k h) through the norm and the residual sum,
    by central differences of the float64 formula: relative error of the
    differences about 1e-8, of the fp32 kernel 1e-5."""
    rows, cols = 4, 40
    x, res = matrix(rows, cols, "f32", 20), matrix(rows, cols, "f32", 21)
    w, c, k = matrix(1, cols, "f32", 22)[0].contiguous(), matrix(rows, cols, "f32", 23), matrix(rows, cols, "f32", 24)
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    ps.opt_rms_norm(x, w, 1e-5, y=y, rstd=rstd, residual=res, h=h, p=0.25, **DRAW)
    dh, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device="cuda")
    ps.opt_rms_norm_backward(c, h, w, rstd, dh, dh_in=k, dx=dx, dweight=dw, p=0.25, **DRAW)
    f = ref.factors(rows, cols, 0.25, **DRAW)

    def loss(xv, rv, wv):
        hv = xv * f + rv
        return (f64(c) * hv * wv / np.sqrt((hv * hv).mean(1, keepdims=True) + 1e-5)).sum() + (f64(k) * hv).sum()

    args = [f64(x), f64(res), f64(w)]
    for i, got in enumerate((dx, dh, dw)):
        want = np.zeros_like(args[i])
        for at in np.ndindex(want.shape):
            up, down = [v.copy() for v in args], [v.copy() for v in args]
            up[i][at] += 1e-4
            down[i][at] -= 1e-4
            want[at] = (loss(*up) - loss(*down)) / 2e-4
        assert np.abs(f64(got) - want).max() <= 2e-5 * np.abs(want).max()


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 4096, 0), (128, 128, 0), (127, 129, 0), (130, 513, 2),
                                           (300, 768, 0), (33, 8, 8), (515, 1030, 0)])
def test_quantize(dtype, block, rows, cols, pad):
    x = matrix(rows, cols, dtype, 30, pad, std=3e-3)
    x[:, :1] *= 500.0
    if rows > 100:
        x[17] = 0.0
        x[40:90] *= 1e-9
    codes, scales = ps.e4m3_storage(rows, cols)
    codes_t, scales_t = ps.e4m3_storage(cols, rows)
    scales.fill_(0xEE)
    scales_t.fill_(0xEE)
    ps.opt_quantize(x, codes, scales, codes_t, scales_t, block_rows=block)
    v = x.float().cpu().numpy()
    for c, s, u, r, n in ((codes, scales, v, rows, cols), (codes_t, scales_t, v.T, cols, rows)):
        e = ref.block_exponents(u.astype(np.float64), block)
        assert (ref.scale_bytes_of(s, r, n) - 127 == e).all()
        assert (c.cpu().numpy() == ref.encode(u, e)).all()
        unused = np.ones(s.numel(), bool)
        unused[ref.tile_places(r, -(-n // 128)).reshape(-1)] = False
        assert (s.cpu().numpy()[unused] == 0xEE).all()
    one, two = ps.e4m3_storage(rows, cols)
    ps.opt_quantize(x, one, two, block_rows=block)             # one orientation alone: the same
    assert torch.equal(one, codes)
    one, two = ps.e4m3_storage(cols, rows)
    ps.opt_quantize(x, codes_t=one, scales_t=two, block_rows=block)
    assert torch.equal(one, codes_t)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_extremes(block):
    """Boundaries of the scale rule, subnormals, the largest fp32, infinities and NaN."""
    x = torch.zeros(256, 256, device="cuda")
    vals = [448.0, np.nextafter(np.float32(448), np.float32(1e9)), 448.0 * 2.0 ** 20, np.finfo(np.float32).max, 1e-45, 1.2e-38,
            2.0 ** -119, 448.0 * 2.0 ** -127, 1.75, 1.7500001, 0.0, -448.0, -7e-5]
    for i, val in enumerate(vals):
        x[i, 0] = float(val)
        x[i, 1] = float(val) / 3
        x[i, 2] = -float(val) / 500
    x[20, 5], x[20, 6] = float("nan"), 2.0
    x[21, 5], x[21, 6] = float("inf"), -3.0
    x[22, 200] = float("-inf")
    codes, scales = ps.e4m3_storage(256, 256)
    codes_t, scales_t = ps.e4m3_storage(256, 256)
    ps.opt_quantize(x, codes, scales, codes_t, scales_t, block_rows=block)
    v = x.cpu().numpy()
    for c, s, u in ((codes, scales, v), (codes_t, scales_t, v.T)):
        e = ref.block_exponents(u.astype(np.float64), block)
        assert (ref.scale_bytes_of(s, 256, 256) - 127 == e).all()
        assert (c.cpu().numpy() & 0x7F == ref.encode(u, e) & 0x7F).all()
        signs = np.isfinite(u)
        assert (c.cpu().numpy() == ref.encode(u, e))[signs].all()


# -------------------------------------------------------------------- matmul
def operand(rows, k, block, seed, std=1.0):
    x = matrix(rows, k, "f32", seed, std=std)
    if rows > 2:
        x[::3] *= 30.0                                        # scales that differ by row
    codes, scales = ps.e4m3_storage(rows, k)
    scales.fill_(0xFF)                                        # NaN wherever the quantizer does not write
    if k:
        ps.opt_quantize(x, codes, scales, block_rows=block)
    return codes, scales


MATMUL_SHAPES = [(1, 1, 1), (1, 16, 16), (1, 4096, 768), (2, 129, 130), (3, 1000, 515), (7, 768, 2304), (16, 128, 128),
                 (17, 300, 1024), (32, 257, 640), (33, 127, 127), (64, 512, 4096), (100, 1, 300), (128, 128, 512),
                 (129, 255, 513), (200, 8, 64), (255, 257, 1100), (256, 256, 256), (300, 2304, 768), (513, 640, 129),
                 (1000, 1031, 77), (2048, 1024, 385)]


@pytest.mark.parametrize("out,addend", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("m,n,k", MATMUL_SHAPES)
def test_matmul(out, addend, m, n, k):
    a, sa = operand(m, k, 1, 40)
    b, sb = operand(n, k, 128 if k % 2 else 1, 41, std=0.05)
    pad = 3 if (m + n) % 2 else 0
    c = matrix(m, n, out, 42, pad=pad) if addend else None
    d = blank(m, n, out, pad)
    ps.opt_matmul(a, sa, b, sb, d, addend=c)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    want = va @ vb.T + (f64(c) if addend else 0.0)
    # a 32-deep step of the tensor core adds its products to the accumulator with errors of at most 2^-23 of
    # the magnitudes that it holds, for each of the products and the accumulator once per step
    bound = (np.abs(va) @ np.abs(vb).T) * 2.0 ** -23 * (k / 32 + 34) + 2.0 ** -24 * np.abs(want)
    within(d, want, out, bound)
    if pad:
        assert (d.as_strided((m, pad), (n + pad, 1), n) == 7).all(), "wrote between the rows"


def test_matmul_exact_sums():
    """Small integers: every partial sum is exact in fp32, so the product is too,
    in every tile, row and column."""
    for m, n, k in ((300, 520, 1000), (5, 700, 4096), (1, 300, 200), (257, 129, 128)):
        g = torch.Generator().manual_seed(m)
        ia, ib = torch.randint(-3, 4, (m, k), generator=g).float(), torch.randint(-3, 4, (n, k), generator=g).float()
        a, sa = ps.e4m3_storage(m, k)
        b, sb = ps.e4m3_storage(n, k)
        ps.opt_quantize(ia.cuda(), a, sa)
        ps.opt_quantize(ib.cuda(), b, sb)
        out = torch.empty(m, n, device="cuda")
        ps.opt_matmul(a, sa, b, sb, out)
        assert torch.equal(out.cpu(), ia @ ib.T)


@pytest.mark.parametrize("m,n,k", [(1, 300, 200), (40, 300, 1000), (300, 520, 77), (700, 1100, 1300)])
def test_matmul_pitch_of_codes(m, n, k):
    """The same bits from rows of any pitch that is a multiple of 16."""
    a, sa = operand(m, k, 1, 48)
    b, sb = operand(n, k, 1, 49)
    want, out = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    ps.opt_matmul(a, sa, b, sb, want)
    for pitch in (-(-k // 16) * 16, -(-k // 16) * 16 + 48):
        wide = []
        for t in (a, b):
            w = torch.full((t.shape[0], pitch), 0x7F, dtype=torch.uint8, device="cuda")[:, :k]      # NaN between the rows
            w.copy_(t)
            wide.append(w)
        ps.opt_matmul(wide[0], sa, wide[1], sb, out)
        assert torch.equal(out, want)


def test_matmul_in_place_sum_depth_zero_and_nan():
    a, sa = operand(70, 200, 1, 50)
    b, sb = operand(90, 200, 1, 51)
    c = matrix(70, 90, "f32", 52)
    want = torch.empty_like(c)
    ps.opt_matmul(a, sa, b, sb, want, addend=c)
    out = c.clone()
    ps.opt_matmul(a, sa, b, sb, out, addend=out)
    assert torch.equal(out, want)
    a0, sa0 = ps.e4m3_storage(70, 0)
    b0, sb0 = ps.e4m3_storage(90, 0)
    ps.opt_matmul(a0, sa0, b0, sb0, out, addend=c)
    assert torch.equal(out, c)
    ps.opt_matmul(a0, sa0, b0, sb0, out)
    assert (out == 0).all()
    a[3, 150] = 0x7F                                          # a NaN code reaches its row and no other
    ps.opt_matmul(a, sa, b, sb, out)
    assert torch.isnan(out[3]).all() and torch.isfinite(out[:3]).all() and torch.isfinite(out[4:]).all()


@pytest.mark.parametrize("m,n", [(150, 150), (150, 5), (60, 150)])
def test_matmul_scales_far_apart(m, n):
    """Row scales from 2^-100 to 2^100 on one side, 2^20 on the other."""
    k = 256
    ia = torch.randint(1, 4, (m, k), generator=torch.Generator().manual_seed(1)).float()
    ib = torch.randint(1, 4, (n, k), generator=torch.Generator().manual_seed(2)).float()
    pa = torch.linspace(-100, 100, m).round()
    a, sa = ps.e4m3_storage(m, k)
    b, sb = ps.e4m3_storage(n, k)
    ps.opt_quantize((ia * torch.exp2(pa)[:, None]).cuda(), a, sa)
    ps.opt_quantize((ib * 2.0 ** 20).cuda(), b, sb)
    out = torch.empty(m, n, device="cuda")
    ps.opt_matmul(a, sa, b, sb, out)
    want = (ia @ ib.T).double() * torch.exp2(pa.double())[:, None] * 2.0 ** 20
    assert torch.equal(out.cpu(), want.float())                # infinite where the product is beyond fp32


# ------------------------------------------------- streams, repetition, graphs
def test_repeats_and_streams_bit_for_bit():
    x, res = matrix(500, 769, "bf16", 60), matrix(500, 769, "bf16", 61)
    w = torch.ones(769, device="cuda")
    dy = matrix(500, 769, "bf16", 62)

    def once(stream=None):
        h, dh = torch.empty_like(x), torch.empty_like(x)
        rstd, dw = torch.empty(500, device="cuda"), torch.empty(769, device="cuda")
        c, s = ps.e4m3_storage(500, 769)
        out = torch.empty(500, 300, device="cuda")
        torch.cuda.synchronize()
        ps.opt_rms_norm(x, w, residual=res, h=h, rstd=rstd, codes=c, scales=s, p=0.1, stream=stream, **DRAW)
        ps.opt_quantize(h, c, s, stream=stream)
        ps.opt_rms_norm_backward(dy, h, w, rstd, dh, dweight=dw, stream=stream)
        ps.opt_matmul(c, s, c[:300], s[:ps.opt_scales_bytes(300, 769)], out, stream=stream)
        torch.cuda.synchronize()
        return h, dh, rstd, dw, c, s, out

    first = once()
    side = torch.cuda.Stream()
    for other in (once(), once(side), once(side.cuda_stream)):
        assert all(torch.equal(p, q) for p, q in zip(first, other))


def test_calls_replay_from_a_graph():
    a, sa = operand(40, 512, 1, 70)
    b, sb = operand(256, 512, 128, 71)
    x = matrix(40, 512, "f32", 72)
    w = torch.ones(512, device="cuda")
    out, want = torch.empty(40, 256, device="cuda"), torch.empty(40, 256, device="cuda")

    def calls(dst):
        ps.opt_rms_norm(x, w, codes=a, scales=sa)
        ps.opt_matmul(a, sa, b, sb, dst)

    calls(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls(out)
    x.mul_(3.0)
    g.replay()
    calls(want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------- guards, aliases, far-off elements
class Guarded:
    """Storage inside a larger allocation of a byte pattern; check() that the
    bytes before and after it still hold the pattern."""
    BAND = 512

    def __init__(self):
        self.kept = []

    def new(self, rows, cols, dtype, pitch=None):
        es = torch.empty(0, dtype=dtype).element_size()
        pitch = pitch or cols
        n = ((rows - 1) * pitch + cols) * es
        flat = torch.full((n + 2 * self.BAND + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        self.kept.append((flat, n, rows, cols, pitch, es))
        return flat[self.BAND:self.BAND + n + (-n) % es].view(dtype).as_strided((rows, cols), (pitch, 1))

    def check(self):
        for flat, n, rows, cols, pitch, es in self.kept:
            inside = torch.zeros_like(flat, dtype=torch.bool)
            body = inside[self.BAND:]
            for r in range(rows):
                body[r * pitch * es:(r * pitch + cols) * es] = True
            assert (flat[~inside] == 0xA5).all(), (rows, cols, pitch)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 5), (3, 769), (129, 264), (20, 4096), (2, 17000), (260, 130)])
def test_nothing_is_written_outside(dtype, rows, cols):
    g = Guarded()
    td, up16 = TD[dtype], lambda n: -(-n // 16) * 16
    x, res, w = matrix(rows, cols, dtype, 80), matrix(rows, cols, dtype, 81), torch.ones(cols, device="cuda")
    h, y, dh, dx = (g.new(rows, cols, td, cols + p) for p in (0, 3, 8, 1))
    rstd, dw = g.new(1, rows, torch.float32).view(-1), g.new(1, cols, torch.float32).view(-1)
    codes, codes_t = g.new(rows, cols, torch.uint8, up16(cols)), g.new(cols, rows, torch.uint8, up16(rows))
    scales = g.new(1, ps.opt_scales_bytes(rows, cols), torch.uint8).view(-1)
    scales_t = g.new(1, ps.opt_scales_bytes(cols, rows), torch.uint8).view(-1)
    work = g.new(1, ps.opt_rms_norm_backward_workspace(rows, cols), torch.uint8).view(-1)
    ps.opt_dropout(x, y, 0.2, residual=res, **DRAW)
    ps.opt_rms_norm(x, w, y=y, rstd=rstd, residual=res, h=h, codes=codes, scales=scales, p=0.2, **DRAW)
    ps.opt_rms_norm_backward(y, h, w, rstd, dh, dx=dx, dweight=dw, p=0.2, workspace=work, **DRAW)
    for block in (1, 128):
        ps.opt_quantize(x, codes, scales, codes_t, scales_t, block_rows=block)
    for out in (torch.float32, torch.bfloat16):
        for pitch in (rows, rows + 16, rows + 3):
            o = g.new(rows, rows, out, pitch)
            ps.opt_matmul(codes, scales, codes, scales, o)                # rows x rows over the columns
        if rows > 1:
            few = g.new(2, rows, out, rows + 1)
            ps.opt_matmul(codes[:2], scales[:ps.opt_scales_bytes(2, cols)], codes, scales, few)
    torch.cuda.synchronize()
    g.check()


@pytest.mark.parametrize("cols", [200, 769, 4096, 20000])
def test_outputs_in_their_inputs_place(cols):
    rows = 37
    x, res, w = matrix(rows, cols, "bf16", 82), matrix(rows, cols, "bf16", 83), torch.ones(cols, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    ps.opt_rms_norm(x, w, residual=res, h=h, y=y, rstd=rstd, p=0.1, **DRAW)
    for place in (0, 1):
        ins = [x.clone(), res.clone()]
        y2 = torch.empty_like(x)
        ps.opt_rms_norm(ins[0], w, residual=ins[1], h=ins[place], y=y2, p=0.1, **DRAW)
        assert torch.equal(ins[place], h) and torch.equal(y2, y)
    dy, dh_in, dh = matrix(rows, cols, "bf16", 84), matrix(rows, cols, "bf16", 85), torch.empty_like(x)
    dw, dw2 = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ps.opt_rms_norm_backward(dy, h, w, rstd, dh, dh_in=dh_in, dweight=dw)
    for place in (0, 1):
        ins = [dy.clone(), dh_in.clone()]
        ps.opt_rms_norm_backward(ins[0], h, w, rstd, ins[place], dh_in=ins[1], dweight=dw2)
        assert torch.equal(ins[place], dh) and torch.equal(dw, dw2)


def test_rows_past_2_31_elements():
    """The last rows of matrices of over 2^31 elements are those of the same rows alone."""
    rows, cols = (1 << 19) + 5, 4104
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = matrix(5, cols, "bf16", 86)
    x.zero_()
    x[-5:] = tail
    w = torch.ones(cols, device="cuda")
    y, y1 = torch.empty_like(x), torch.empty_like(tail)
    ps.opt_rms_norm(x, w, y=y)
    ps.opt_rms_norm(tail, w, y=y1)
    assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
    ps.opt_rms_norm_backward(x, x, w, torch.ones(rows, device="cuda"), y)
    ps.opt_rms_norm_backward(tail, tail, w, torch.ones(5, device="cuda"), y1)
    assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
    del y
    c, s = ps.e4m3_storage(rows, cols)
    c1, s1 = ps.e4m3_storage(5, cols)
    ps.opt_quantize(x, c, s)
    ps.opt_quantize(tail, c1, s1)
    assert torch.equal(c[-5:], c1)
    assert (ref.scale_bytes_of(s, rows, cols)[-5:] == ref.scale_bytes_of(s1, 5, cols)).all()


def test_product_of_over_2_31_elements():
    m, n = 70001, 40000
    a, sa = operand(m, 128, 1, 87)
    b, sb = operand(n, 128, 1, 88)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ps.opt_matmul(a, sa, b, sb, out)
    vb = ref.values(b, sb)
    e = ref.scale_bytes_of(sa, m, 128) - 127
    for r in (0, 55001, m - 1):
        row = a[r].cpu().view(torch.float8_e4m3fn).double().numpy() * 2.0 ** float(e[r, 0])
        bound = (np.abs(vb) @ np.abs(row)) * 2.0 ** -23 * 38
        within(out[r], vb @ row, "bf16", bound)


@pytest.mark.parametrize("m,n,k", [(40, 256, 1024), (300, 200, 700), (1024, 2048, 256)])
def test_wait_drill(m, n, k):
    """A product whose waits run out reports it, leaves its output alone, and
    changes nothing for the next one.  (One shape per form: split, single CTAs,
    pairs.)"""
    a, sa = operand(m, k, 1, 90)
    b, sb = operand(n, k, 1, 91)
    out, want = blank(m, n, "f32"), torch.empty(m, n, device="cuda")
    assert ps.opt_layer_status() == 0
    ps.opt_matmul(a, sa, b, sb, out, wait_drill=True)
    assert ps.opt_layer_status() == ps.OPT_FLAG_WAIT_TIMEOUT and (out == 7).all()
    assert ps.opt_layer_status() == 0
    ps.opt_matmul(a, sa, b, sb, want)
    ps.opt_matmul(a, sa, b, sb, out)
    assert torch.equal(out, want) and ps.opt_layer_status() == 0


def test_status_is_clear():
    """Every kernel of the tests above ran to completion."""
    assert ps.opt_layer_status() == 0
