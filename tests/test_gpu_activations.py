"""GPU tests of the gated activation, the heads' norm with rotation, their gradients
and kept activations against definitions in float64 (tests/activation_reference.py,
which derives the bounds), at the sizes, layouts and values where they can go wrong,
and of the gradients against differences."""
import numpy as np
import pytest
import torch

import activation_reference as act
import layer_reference as ref
import precision_states_gb300 as ps
from test_gpu_layer import TD, Guarded, blank, f64, matrix
from test_gpu_layer import within as within_units

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
KINDS = ["silu", "gelu_tanh", "gelu", "relu"]


def within(got, want, dtype, d):
    """As there, and below the type's normal numbers: an output there is off by half of the
    smallest subnormal (2^-134 in BF16, 2^-150 in fp32), and a product that passes through
    fp32's subnormals on the way by 2^-150 times the factors that follow, here below 2^9 (2^-140
    with two of them)."""
    within_units(got, want, dtype, d + 2.0 ** -140 + (2.0 ** -135 if dtype == "bf16" else 2.0 ** -151))


def storage(rows, cols):
    codes, scales = ps.e4m3_storage(rows, cols)
    scales.fill_(0xEE)
    return codes, scales


def kept(x):
    pair = storage(*x.shape)
    ps.opt_quantize(x, *pair)
    return pair


def as_values(x):
    """float64 values of a matrix or a kept one."""
    return ref.values(*x) if isinstance(x, tuple) else f64(x)


def spread(rows, cols, dtype, seed, pad=0, shift=0):
    """Gates over the whole range of the activation: mostly unit values, some near 0 and
    some far out."""
    x = matrix(rows, cols, dtype, seed, pad, shift)
    x[:, ::7] *= 30.0
    x[:, 3::11] *= 1e-3
    return x


# ---------------------------------------------------------------- dequantize
SHAPES = [(1, 1, 0), (1, 4096, 0), (3, 8, 0), (128, 128, 0), (127, 129, 0), (130, 513, 2), (300, 768, 8), (33, 2305, 3),
          (515, 1030, 0), (700, 24, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_dequantize(dtype, rows, cols, pad):
    """Values are exact in fp32 and rounded once in BF16; the turned operand is the
    quantizer's of the values, transposed."""
    x = matrix(rows, cols, "f32", 1, std=3e-3)
    x[:, :1] *= 500.0
    if rows > 100:
        x[17] = 0.0
        x[40:90] *= 1e-9
    pair = kept(x)
    v = ref.values(*pair)
    assert (v.astype(np.float32) == v).all()
    want = torch.from_numpy(v).float().to(TD[dtype]).cuda()
    out, (ct, st) = blank(rows, cols, dtype, pad), storage(cols, rows)
    ps.opt_dequantize(*pair, x=out, codes_t=ct, scales_t=st)
    assert torch.equal(out, want)
    act.check_kept(ct, st, v.T.astype(np.float32))
    assert act.untouched(st, cols, rows, 0xEE)
    if pad and rows > 1:
        assert (out.as_strided((rows - 1, pad), (cols + pad, 1), cols) == 7).all(), "wrote between the rows"
    out2, (c2, s2) = blank(rows, cols, dtype), storage(cols, rows)      # each alone: the same
    ps.opt_dequantize(*pair, x=out2)
    ps.opt_dequantize(*pair, codes_t=c2, scales_t=s2)
    assert torch.equal(out2, want) and torch.equal(c2, ct) and torch.equal(s2, st)


def test_dequantize_every_code_and_scale():
    """All 256 codes with all 256 scale bytes: subnormal and overflowing values, NaN codes
    and the NaN scale; a column then holds scales of every size."""
    codes, scales = ps.e4m3_storage(256, 256)
    codes.copy_(torch.arange(256, dtype=torch.uint8, device="cuda")[None, :].expand(256, 256))
    tiles = np.zeros(scales.numel(), np.uint8)
    for b in range(2):
        tiles[ref.tile_places(256, 2)[:, b]] = np.arange(256)
    scales.copy_(torch.from_numpy(tiles))
    c = codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    with np.errstate(all="ignore"):
        v = (c * 2.0 ** (np.arange(256.0)[:, None] - 127)).astype(np.float32)
    v[255] = np.nan
    out = blank(256, 256, "f32")
    ct, st = storage(256, 256)
    ps.opt_dequantize(codes, scales, x=out, codes_t=ct, scales_t=st)
    got = out.cpu().numpy()
    assert (np.isnan(got) == np.isnan(v)).all() and (got[~np.isnan(v)] == v[~np.isnan(v)]).all()
    act.check_kept(ct, st, np.ascontiguousarray(v.T))
    for lo, hi in ((100, 140), (0, 12), (240, 255)):                   # and without the far-off rows
        sub = codes[lo:hi].contiguous()
        ss = storage(hi - lo, 256)[1]
        t2 = np.zeros(ss.numel(), np.uint8)
        for b in range(2):
            t2[ref.tile_places(hi - lo, 2)[:, b]] = np.arange(lo, hi)
        ss.copy_(torch.from_numpy(t2))
        ct, st = storage(256, hi - lo)
        ps.opt_dequantize(sub, ss, codes_t=ct, scales_t=st)
        act.check_kept(ct, st, np.ascontiguousarray(v[lo:hi].T))


# --------------------------------------------------------------------- gated
GATED_SHAPES = [(1, 1, 0, 0), (1, 14336, 0, 0), (3, 8, 0, 0), (2, 127, 0, 0), (5, 129, 3, 1), (130, 769, 0, 0), (67, 768, 8, 0),
                (9, 2304, 0, 0), (4, 5001, 1, 1), (300, 33, 0, 1), (513, 264, 0, 0), (70001, 1, 0, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", GATED_SHAPES)
def test_gated(dtype, rows, cols, pad, shift):
    kind, has_up = KINDS[(rows + cols) % 4], (rows + 2 * cols) % 3 > 0
    if rows > 1000:
        kind = "silu"
    g = spread(rows, cols, dtype, 4, pad, shift)
    u = matrix(rows, cols, dtype, 5, pad) if has_up else None
    y, pair, gk, uk = blank(rows, cols, dtype, pad), storage(rows, cols), storage(rows, cols), storage(rows, cols)
    ps.opt_gated(g, u, activation=kind, y=y, codes=pair[0], scales=pair[1], gate_kept=gk, up_kept=uk if has_up else None)
    f, _, d, _ = act.activation(f64(g), kind)
    uv = f64(u) if has_up else 1.0
    want, d = f * uv, d * np.abs(uv) + E24 * np.abs(f * uv)
    within(y, want, dtype, d)
    act.check_codes(*pair, want, d)
    act.check_kept(*gk, g.float().cpu().numpy())
    if has_up:
        act.check_kept(*uk, u.float().cpu().numpy())
    for p in (pair, gk):
        assert act.untouched(p[1], rows, cols, 0xEE)
    if pad and rows > 1:
        assert (y.as_strided((rows - 1, pad), (cols + pad, 1), cols) == 7).all(), "wrote between the rows"
    y2 = blank(rows, cols, dtype)                                      # one output alone: the same
    ps.opt_gated(g, u, activation=kind, y=y2)
    assert torch.equal(y2, y)
    ps.opt_gated(g, u, activation=kind, y=g)                           # in the gate's place
    assert torch.equal(g, y)


@pytest.mark.parametrize("kind", KINDS)
def test_every_kind_over_the_range(kind):
    """Gates from -120 to 120 and the type's largest: no overflow on the way; gradients from
    plain inputs."""
    g = torch.cat([torch.linspace(-120, 120, 4093, device="cuda"), torch.tensor([3e38, -3e38, 0.0], device="cuda")])[None]
    u = matrix(1, 4096, "f32", 6)
    dy = matrix(1, 4096, "f32", 7)
    y, dg, du = blank(1, 4096, "f32"), blank(1, 4096, "f32"), blank(1, 4096, "f32")
    ps.opt_gated(g, activation=kind, y=y)
    f, df, d, dd = act.activation(f64(g), kind)
    within(y, f, "f32", d)
    assert torch.isfinite(y).all()
    ps.opt_gated_backward(dy, g, u, activation=kind, dgate=dg, dup=du)
    w = f64(dy) * f64(u)
    finite = np.abs(f64(dy) * f) < 3e38
    within(dg, w * df, "f32", np.abs(w) * dd + 3 * E24 * np.abs(w * df))
    want = f64(dy) * f
    err = np.abs(f64(du) - want)[finite]
    assert (err <= (E24 * np.abs(want) + 2 * (np.abs(f64(dy)) * d + E24 * np.abs(want)))[finite]).all()


def test_gated_special_values():
    inf, nan = float("inf"), float("nan")
    for dtype in ("bf16", "f32"):
        g = torch.tensor([[nan, inf, -inf, 1.0, 1.0, 0.0, -0.0, 2.0]], device="cuda").to(TD[dtype])
        u = torch.tensor([[1.0, 1.0, 1.0, nan, inf, 3.0, inf, 0.0]], device="cuda").to(TD[dtype])
        for kind in KINDS:
            y, pair, gk = blank(1, 8, dtype), storage(1, 8), storage(1, 8)
            ps.opt_gated(g, u, activation=kind, y=y, codes=pair[0], scales=pair[1], gate_kept=gk)
            v = y.float()[0].tolist()
            assert np.isnan(v[0]) and v[1] == inf and np.isnan(v[3]) and v[4] == inf and v[5] == 0 and np.isnan(v[6]) and v[7] == 0
            assert v[2] == 0 if kind == "relu" else np.isnan(v[2])
            assert [int(c) & 0x7F == 0x7F for c in pair[0][0].tolist()] == [not np.isfinite(x) for x in v]
            assert [int(c) & 0x7F == 0x7F for c in gk[0][0].tolist()] == [True] * 3 + [False] * 5
            dg = blank(1, 8, dtype)
            ps.opt_gated_backward(torch.ones_like(g), g, u, activation=kind, dgate=dg)
            assert torch.isnan(dg[0, 0]) and torch.isnan(dg[0, 3]) and dg[0, 5] == 3.0 * (0.5 if kind != "relu" else 0.0)


@pytest.mark.parametrize("source", ["plain", "kept"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift", GATED_SHAPES + [(257, 640, 0, 0), (128, 512, 64, 0)])
def test_gated_backward(dtype, source, rows, cols, pad, shift):
    kind, has_up = KINDS[(rows + cols) % 4], (rows + 2 * cols) % 3 > 0
    if rows > 1000:
        kind = "silu"
    g = spread(rows, cols, dtype, 8, pad, shift)
    u = matrix(rows, cols, dtype, 9, pad) if has_up else None
    dy = matrix(rows, cols, dtype, 10, pad, shift, std=1e-2)
    gs, us = (kept(g), kept(u) if has_up else None) if source == "kept" else (g, u)
    names = ["dgate", "dup"] if has_up else ["dgate"]
    plain = {n: blank(rows, cols, dtype, pad) for n in names}
    coded = {n + "_codes": storage(rows, cols) for n in names}
    turned = {n + "_codes_t": storage(cols, rows) for n in names + ["y"]}
    ps.opt_gated_backward(dy, gs, us, activation=kind, **plain, **coded, **turned)
    gv, uv, dv = as_values(gs), as_values(us) if has_up else 1.0, f64(dy)
    f, df, d, dd = act.activation(gv, kind)
    want = {"dgate": dv * df * uv, "dup": dv * f, "y": f * uv}
    off = {"dgate": np.abs(dv * uv) * dd + 3 * E24 * np.abs(want["dgate"]), "dup": np.abs(dv) * d + 2 * E24 * np.abs(want["dup"]),
           "y": np.abs(uv) * d + 2 * E24 * np.abs(want["y"])}
    for n in names:
        within(plain[n], want[n], dtype, off[n])
        act.check_codes(*coded[n + "_codes"], want[n], off[n])
        assert act.untouched(coded[n + "_codes"][1], rows, cols, 0xEE)
        if pad and rows > 1:
            assert (plain[n].as_strided((rows - 1, pad), (cols + pad, 1), cols) == 7).all(), "wrote between the rows"
    for n in names + ["y"]:
        act.check_codes(*turned[n + "_codes_t"], want[n].T, off[n].T)
        assert act.untouched(turned[n + "_codes_t"][1], cols, rows, 0xEE)
    # without the transposed outputs, and each alone: the same bits
    plain2, coded2 = {n: blank(rows, cols, dtype) for n in names}, {n + "_codes": storage(rows, cols) for n in names}
    ps.opt_gated_backward(dy, gs, us, activation=kind, **plain2, **coded2)
    for n in names:
        assert torch.equal(plain2[n], plain[n])
        for p, q in zip(coded2[n + "_codes"], coded[n + "_codes"]):
            assert torch.equal(p, q)
    one = storage(cols, rows)
    for n in names + ["y"]:
        ps.opt_gated_backward(dy, gs, us, activation=kind, **{n + "_codes_t": one})
        assert torch.equal(one[0], turned[n + "_codes_t"][0]) and torch.equal(one[1], turned[n + "_codes_t"][1])


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("cols,pad,shift", [(512, 0, 0), (769, 0, 1), (130, 3, 0)])
def test_gated_outputs_in_their_inputs_place(turn, cols, pad, shift):
    rows = 300
    g, u, dy = (matrix(rows, cols, "bf16", 20 + i, pad, shift) for i in range(3))
    want = [blank(rows, cols, "bf16"), blank(rows, cols, "bf16")]
    t = {"y_codes_t": storage(cols, rows)} if turn else {}
    ps.opt_gated_backward(dy, g, u, dgate=want[0], dup=want[1], **t)
    for first, second in (("g", "u"), ("u", "g"), ("dy", "u"), ("g", "dy")):
        m = dict(g=g.clone(), u=u.clone(), dy=dy.clone())
        if pad or shift:
            for k, v in m.items():
                wide = torch.zeros(rows * (cols + pad) + shift, dtype=torch.bfloat16, device="cuda")
                m[k] = wide[shift:].view(rows, cols + pad)[:, :cols]
                m[k].copy_(v)
        ps.opt_gated_backward(m["dy"], m["g"], m["u"], dgate=m[first], dup=m[second], **t)
        assert torch.equal(m[first], want[0]) and torch.equal(m[second], want[1])


def test_gated_backward_against_differences():
    """The gradient of sum(c f(g) u) by central differences in float64."""
    g, u, c = (matrix(3, 40, "f32", 30 + i) for i in range(3))
    for kind in ("silu", "gelu_tanh", "gelu"):
        dg, du = torch.empty_like(g), torch.empty_like(g)
        ps.opt_gated_backward(c, g, u, activation=kind, dgate=dg, dup=du)
        f = lambda x: act.activation(x, kind)[0]  # noqa: E731
        gv, uv, cv = f64(g), f64(u), f64(c)
        want = cv * uv * (f(gv + 1e-5) - f(gv - 1e-5)) / 2e-5
        assert np.abs(f64(dg) - want).max() <= 1e-6 * np.abs(want).max()
        assert np.abs(f64(du) - cv * f(gv)).max() <= 1e-6 * np.abs(cv * f(gv)).max()


# --------------------------------------------------------------------- heads
def tables(positions, rot, base=1e4):
    angle = np.arange(positions)[:, None] * base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return (torch.from_numpy(np.cos(angle)).float().cuda(), torch.from_numpy(np.sin(angle)).float().cuda()) if rot else (None, None)


def places(rows, table, seed):
    return torch.randint(0, table, (rows,), generator=torch.Generator().manual_seed(seed)).cuda()


def heads_of(t, dim):
    return t.reshape(t.shape[0], -1, dim)


# rows, query heads, key heads, dim, rot, interleaved, padding of the rows
HEADS = [(1, 32, 8, 128, 128, False, 0), (1, 1, 0, 64, 64, True, 0), (5, 3, 1, 64, 32, True, 8), (130, 12, 12, 64, 64, False, 0),
         (67, 7, 7, 32, 32, False, 8), (33, 5, 2, 96, 96, False, 0), (40, 9, 3, 80, 80, False, 0), (9, 4, 4, 256, 128, False, 0),
         (17, 3, 3, 160, 160, True, 0), (21, 2, 1, 192, 64, False, 0), (300, 17, 3, 16, 16, False, 0), (50, 33, 1, 8, 8, True, 0),
         (11, 3, 2, 128, 0, False, 0), (65, 2, 2, 128, 120, True, 0),
         # heads of any size and place
         (1, 2, 1, 33, 32, False, 0), (40, 5, 3, 100, 100, False, 0), (23, 3, 2, 64, 64, False, 3), (31, 2, 2, 64, 24, False, 0),
         (7, 1, 1, 1, 0, False, 0), (12, 2, 1, 2, 2, True, 1), (3, 1, 2, 1024, 1024, True, 0), (5, 2, 0, 300, 150, False, 0),
         (2000, 3, 1, 40, 40, False, 0), (700, 1, 1, 50, 26, True, 0)]
# by single elements: up to 64, 128 and 256 of them, and rows that begin anywhere
HEADS += [(31, 9, 2, 255, 250, False, 0), (33, 3, 3, 130, 64, True, 0), (20, 4, 1, 256, 256, False, 1), (9, 11, 5, 63, 62, True, 0),
          (130, 2, 2, 129, 0, False, 0), (5, 17, 2, 128, 64, False, 5), (4, 1, 0, 257, 256, True, 0)]
# whole chunks of which any even part is rotated
PARTS = [(33, 5, 2, 64, 24, False, 0), (40, 9, 3, 80, 40, False, 8), (300, 3, 1, 128, 2, False, 0), (9, 2, 2, 256, 250, False, 0),
         (70, 17, 3, 16, 14, False, 0), (5, 33, 1, 8, 6, False, 0), (21, 6, 1, 24, 18, False, 0), (3001, 3, 2, 96, 90, False, 0),
         (65, 2, 2, 128, 118, True, 0), (50, 12, 1, 8, 2, True, 0), (130, 4, 2, 112, 54, True, 8), (1, 7, 2, 200, 100, False, 0)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,hq,hk,dim,rot,interleaved,pad", HEADS + PARTS)
def test_head_norm(dtype, wdtype, rows, hq, hk, dim, rot, interleaved, pad):
    cos, sin = tables(97, rot)
    at = places(rows, 97, 1) if rot else None
    how = dict(eps=1e-5, cos=cos, sin=sin, positions=at, interleaved=interleaved)
    side, more, checks = {}, {}, []
    for name, heads, seed in (("q", hq, 2), ("k", hk, 3)):
        if heads == 0:
            continue
        x = matrix(rows, heads * dim, dtype, seed, pad, std=2.0)
        w = (1 + 0.2 * matrix(1, dim, "f32", seed + 10)[0]).to(TD[wdtype])
        out, pair = blank(rows, heads * dim, dtype, pad), storage(rows, heads * dim)
        side[name] = (x, w, out, pair)
        c, s = (t.double().cpu().numpy()[at.cpu().numpy()] if rot else None for t in (cos, sin))
        y, d = act.head_norm(f64(heads_of(x, dim)), f64(w), 1e-5, c, s, rot, interleaved)
        checks.append((out, y.reshape(rows, -1), d.reshape(rows, -1), x.clone(), pair))
    if hk:
        x, w, out, pair = side["k"]
        more = dict(k=x, k_weight=w, k_out=out, k_kept=pair)
    x, w, out, pair = side["q"]
    ps.opt_head_norm(x, w, out, q_kept=pair, **more, **how)
    for out, y, d, x, pair in checks:
        within(out, y, dtype, d)
        act.check_kept(*pair, x.float().cpu().numpy())
        assert act.untouched(pair[1], rows, x.shape[1], 0xEE)
        if pad and rows > 1:
            assert (out.as_strided((rows - 1, pad), (x.shape[1] + pad, 1), x.shape[1]) == 7).all(), "wrote between the rows"
    # in the inputs' place, without keeping: the same bits
    for name, (x, w, out, pair) in side.items():
        ps.opt_head_norm(x, w, x, **how)
        assert torch.equal(x, out)


@pytest.mark.parametrize("source", ["plain", "kept"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,hq,hk,dim,rot,interleaved,pad", HEADS + PARTS)
def test_head_norm_backward(dtype, wdtype, source, rows, hq, hk, dim, rot, interleaved, pad):
    cos, sin = tables(97, rot)
    at = places(rows, 97, 1) if rot else None
    how = dict(eps=1e-5, cos=cos, sin=sin, positions=at, interleaved=interleaved)
    args, checks = {}, []
    for name, heads, seed in (("q", hq, 4), ("k", hk, 5)):
        if heads == 0:
            continue
        x = matrix(rows, heads * dim, dtype, seed, pad, std=2.0)
        x = kept(x) if source == "kept" else x
        dout = matrix(rows, heads * dim, dtype, seed + 10, pad, std=0.1)
        w = (1 + 0.2 * matrix(1, dim, "f32", seed + 20)[0]).to(TD[wdtype])
        dx, dw = blank(rows, heads * dim, dtype, pad), torch.full((dim,), 7.0, device="cuda")
        args.update({name: x, "d%s_out" % name: dout, name + "_weight": w, "d" + name: dx, "d%s_weight" % name: dw})
        c, s = (t.double().cpu().numpy()[at.cpu().numpy()] if rot else None for t in (cos, sin))
        want = act.head_norm_backward(f64(heads_of(dout, dim)), as_values(x).reshape(rows, heads, dim), f64(w), 1e-5, c, s, rot, interleaved)
        checks.append((dx, dw, want, heads))
    ps.opt_head_norm_backward(**args, **how)
    for dx, dw, (want, d, wanted, size), heads in checks:
        within(dx, want.reshape(rows, -1), dtype, d.reshape(rows, -1))
        # at most every term after another, each with the roundings that rstd and g carry
        assert (np.abs(f64(dw) - wanted) <= E24 * (rows * heads + dim / 32 + 30) * size).all()
        if pad and rows > 1:
            assert (dx.as_strided((rows - 1, pad), (dx.shape[1] + pad, 1), dx.shape[1]) == 7).all(), "wrote between the rows"
    # without the weights' gradients, and in dout's place: the same bits
    for name in ("q", "k") if hk else ("q",):
        dout = args["d%s_out" % name]
        ps.opt_head_norm_backward(dout, args[name], args[name + "_weight"], dout, **how)
        assert torch.equal(dout, args["d" + name])


def test_head_norm_backward_against_differences():
    rows, heads, dim, rot = 3, 2, 24, 16
    x, c = matrix(rows, heads * dim, "f32", 40), matrix(rows, heads * dim, "f32", 41)
    w = matrix(1, dim, "f32", 42)[0].contiguous()
    cos, sin = tables(50, rot)
    at = places(rows, 50, 2)
    cv, sv = (t.double().cpu().numpy()[at.cpu().numpy()] for t in (cos, sin))
    for interleaved in (False, True):
        dx, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
        ps.opt_head_norm_backward(c, x, w, dx, dq_weight=dw, cos=cos, sin=sin, positions=at, interleaved=interleaved)

        def loss(xv, wv):
            return (act.head_norm(xv, wv, 1e-5, cv, sv, rot, interleaved)[0] * f64(heads_of(c, dim))).sum()

        args = [f64(heads_of(x, dim)), f64(w)]
        for i, got in enumerate((heads_of(dx, dim), dw)):
            want = np.zeros_like(args[i])
            for place in np.ndindex(want.shape):
                up, down = [v.copy() for v in args], [v.copy() for v in args]
                up[i][place] += 1e-5
                down[i][place] -= 1e-5
                want[place] = (loss(*up) - loss(*down)) / 2e-5
            assert np.abs(f64(got) - want).max() <= 2e-6 * np.abs(want).max()


@pytest.mark.parametrize("dim,shift", [(128, 0), (64, 1)])
def test_heads_special_rows_and_positions(dim, shift):
    """Rows of zeros, infinities and NaN reach their own heads and no others; a position
    outside the tables makes the rotated elements NaN and reads nothing."""
    rows, heads, rot = 8, 4, dim // 2
    cos, sin = tables(10, rot)
    x = matrix(rows, heads * dim, "f32", 50, 0, shift)
    x[1, :dim] = 0.0
    x[2, dim + 3] = float("nan")
    x[3, 5] = float("inf")
    x[4, :dim] = 1e25                                                  # squares overflow fp32
    at = torch.tensor([0, 1, 2, 3, 4, -1, 10, 9], device="cuda")
    far = at.clone()
    far[5], far[6] = -(1 << 62), (1 << 62)
    w = torch.ones(dim, device="cuda")
    y, ok = torch.empty_like(x), torch.empty_like(x)
    ps.opt_head_norm(x, w, y, cos=cos, sin=sin, positions=at)
    ps.opt_head_norm(x, w, ok, cos=cos, sin=sin, positions=at.clamp(0, 9))
    h = heads_of(y, dim)
    assert (h[1, 0] == 0).all() and torch.isfinite(h[1, 1:]).all()
    assert torch.isnan(h[2, 1]).all() and torch.isfinite(h[2, 0]).all() and torch.isfinite(h[2, 2:]).all()
    assert (h[4, 0] == 0).all()
    for r in (5, 6):
        assert torch.isnan(h[r, :, :rot]).all() and torch.equal(h[r, :, rot:], heads_of(ok, dim)[r, :, rot:])
    for r in (0, 7):
        assert torch.equal(y[r], ok[r])
    y2 = torch.empty_like(x)
    ps.opt_head_norm(x, w, y2, cos=cos, sin=sin, positions=far)
    assert torch.equal(torch.nan_to_num(y2, 7), torch.nan_to_num(y, 7))
    dx, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    x = matrix(rows, heads * dim, "f32", 51, 0, shift)
    ps.opt_head_norm_backward(torch.ones_like(x), x, w, dx, dq_weight=dw, cos=cos, sin=sin, positions=at)
    assert torch.isnan(dx[5:7]).all() and torch.isfinite(dx[:5]).all() and torch.isfinite(dx[7]).all()
    assert torch.isnan(dw[:rot]).all()


@pytest.mark.parametrize("dim,rot,interleaved", [(128, 64, False), (64, 24, False), (64, 20, True), (100, 50, False)])
def test_tables_at_any_place_and_infinities_past_the_rotated(dim, rot, interleaved):
    """Tables that start on 4 bytes; an infinity behind the rotated elements stays out of the
    weight's gradient of the others."""
    rows, heads = 37, 3
    cos, sin = tables(rows, rot)
    odd = [torch.empty(t.numel() + 1, device="cuda")[1:].view(t.shape).copy_(t) for t in (cos, sin)]
    for dtype in ("bf16", "f32"):
        x, d = matrix(rows, heads * dim, dtype, 60), matrix(rows, heads * dim, dtype, 61)
        d[5, dim + rot] = float("inf")
        w = torch.ones(dim, device="cuda")
        got = []
        for c, s in ((cos, sin), odd):
            y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(dim, device="cuda")
            ps.opt_head_norm(x, w, y, cos=c, sin=s, interleaved=interleaved)
            ps.opt_head_norm_backward(d, x, w, dx, dq_weight=dw, cos=c, sin=s, interleaved=interleaved)
            got.append((y, torch.nan_to_num(dx, 7.0), dw))
        assert all(torch.equal(a, b) for a, b in zip(*got))
        dw = got[0][2]
        assert torch.isinf(dw[rot]) and torch.isfinite(dw[:rot]).all() and torch.isfinite(dw[rot + 1:]).all()


def test_row_numbers_as_positions_and_shapes_of_heads():
    """Without positions a row's number is its place; heads as a third dimension, inside a
    projection's rows, and as a batch of sequences are the same heads."""
    rows, hq, hk, dim = 30, 4, 2, 64
    x = matrix(rows, (hq + 2 * hk) * dim, "bf16", 60)
    cos, sin = tables(rows, dim)
    w = torch.ones(dim, device="cuda")
    q, k = x[:, :hq * dim], x[:, hq * dim:(hq + hk) * dim]
    want = [torch.empty(rows, n * dim, dtype=torch.bfloat16, device="cuda") for n in (hq, hk)]
    ps.opt_head_norm(q, w, want[0], k, w, want[1], cos=cos, sin=sin, positions=torch.arange(rows, device="cuda"))
    got = [torch.empty_like(t) for t in want]
    ps.opt_head_norm(q, w, got[0], k, w, got[1], cos=cos, sin=sin)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    three = [q.unflatten(1, (hq, dim)), k.unflatten(1, (hk, dim))]
    got = [torch.empty(rows, n, dim, dtype=torch.bfloat16, device="cuda") for n in (hq, hk)]
    ps.opt_head_norm(three[0], w, got[0], three[1], w, got[1], cos=cos, sin=sin)
    assert all(torch.equal(a.flatten(1), b) for a, b in zip(got, want))
    batch = torch.empty(5, 6, hq, dim, dtype=torch.bfloat16, device="cuda")
    ps.opt_head_norm(three[0].contiguous().view(5, 6, hq, dim), w, batch, cos=cos, sin=sin)
    assert torch.equal(batch.view(rows, -1), want[0])
    with pytest.raises(ps.OptError) as e:                              # more rows than positions
        ps.opt_head_norm(q, w, want[0], cos=cos[:29], sin=sin[:29])
    assert e.value.status == ps.OPT_EINVAL


def test_no_rows_and_no_columns():
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 7.0, device="cuda")
    none = torch.empty(0, 128, device="cuda")
    ps.opt_head_norm(none, w, none)
    ps.opt_head_norm_backward(none, none, w, none, dq_weight=dw)
    assert (dw == 0).all()
    q, k = matrix(3, 64, "f32", 210), torch.empty(3, 0, device="cuda")       # no key heads
    dw.fill_(7.0)
    ps.opt_head_norm(q, w, q, k, w, k)
    ps.opt_head_norm_backward(q, q, w, q, k, k, w, k, dk_weight=dw)
    assert (dw == 0).all()
    for shape in ((0, 64), (5, 0)):
        x = torch.empty(*shape, device="cuda")
        c, s = ps.e4m3_storage(*shape)
        ps.opt_gated(x, x, y=x, codes=c, scales=s)
        ps.opt_gated_backward(x, x, x, dgate=x, dup=x)
        ps.opt_dequantize(c, s, x=x)


# ------------------------------------------- guards, far-off elements, repetition
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 5), (3, 769), (129, 264), (20, 4096), (260, 130)])
def test_nothing_is_written_outside(dtype, rows, cols):
    g = Guarded()
    td, up16 = TD[dtype], lambda n: -(-n // 16) * 16  # noqa: E731

    def pair(r, c):
        return g.new(r, c, torch.uint8, up16(c)), g.new(1, ps.opt_scales_bytes(r, c), torch.uint8).view(-1)

    x, u, dy = (matrix(rows, cols, dtype, 70 + i) for i in range(3))
    y, dg, du, out = (g.new(rows, cols, td, cols + p) for p in (3, 8, 1, 0))
    gk, uk, yk = pair(rows, cols), pair(rows, cols), pair(rows, cols)
    ps.opt_gated(x, u, y=y, codes=yk[0], scales=yk[1], gate_kept=gk, up_kept=uk)
    t = {n: pair(cols, rows) for n in ("dgate_codes_t", "dup_codes_t", "y_codes_t")}
    n = {n: pair(rows, cols) for n in ("dgate_codes", "dup_codes")}
    for src in ((gk, uk), (x, u)):
        ps.opt_gated_backward(dy, *src, dgate=dg, dup=du, **n, **t)
        ps.opt_gated_backward(dy, *src, dgate=dg, dup=du, **n)
    ps.opt_dequantize(*gk, x=out, codes_t=t["y_codes_t"][0], scales_t=t["y_codes_t"][1])
    ps.opt_dequantize(*gk, x=out)
    torch.cuda.synchronize()
    g.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq,hk,dim", [(1, 3, 1, 64), (37, 5, 2, 128), (20, 3, 2, 96), (9, 2, 1, 33), (5, 33, 3, 8)])
def test_heads_write_nothing_outside(dtype, rows, hq, hk, dim):
    g = Guarded()
    rot = dim // 4 * 2
    cos, sin = tables(rows, rot)
    w = torch.ones(dim, device="cuda")
    new = lambda h, p: g.new(rows, h * dim, TD[dtype], h * dim + p)  # noqa: E731
    pair = lambda h: (g.new(rows, h * dim, torch.uint8, -(-h * dim // 16) * 16),  # noqa: E731
                      g.new(1, ps.opt_scales_bytes(rows, h * dim), torch.uint8).view(-1))
    q, k = matrix(rows, hq * dim, dtype, 80), matrix(rows, hk * dim, dtype, 81)
    for p in (0, 3):
        qk, kk = pair(hq), pair(hk)
        ps.opt_head_norm(q, w, new(hq, p), k, w, new(hk, p), cos=cos, sin=sin, q_kept=qk, k_kept=kk)
        dw = [g.new(1, dim, torch.float32).view(-1) for _ in range(2)]
        work = g.new(1, ps.opt_head_norm_backward_workspace(rows, hq, hk, dim), torch.uint8).view(-1)
        for qs, ks in ((q, k), (qk, kk)):
            ps.opt_head_norm_backward(q, qs, w, new(hq, p), k, ks, w, new(hk, p), *dw, cos=cos, sin=sin, workspace=work)
    torch.cuda.synchronize()
    g.check()


def test_rows_past_2_31_elements():
    """The last rows of matrices of over 2^31 elements are those of the same rows alone."""
    rows, cols = (1 << 19) + 5, 4104
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = matrix(5, cols, "bf16", 90)
    x[-5:] = tail
    y, y1 = torch.empty_like(x), torch.empty_like(tail)
    ps.opt_gated(x, x, y=y)
    ps.opt_gated(tail, tail, y=y1)
    assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
    c, s = ps.e4m3_storage(rows, cols)
    c1, s1 = ps.e4m3_storage(5, cols)
    ps.opt_gated(x, codes=c, scales=s)
    ps.opt_gated(tail, codes=c1, scales=s1)
    assert torch.equal(c[-5:], c1)
    ps.opt_gated_backward(x, (c, s), dgate=y)
    ps.opt_gated_backward(tail, (c1, s1), dgate=y1)
    assert torch.equal(y[-5:], y1)
    ps.opt_dequantize(c, s, x=y)
    ps.opt_dequantize(c1, s1, x=y1)
    assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
    w = torch.ones(1026, device="cuda")[:513].contiguous()
    for dim in (8, 513):                                               # whole chunks, and any
        w = torch.ones(dim, device="cuda")
        ps.opt_head_norm(x, w, y)
        ps.opt_head_norm(tail, w, y1)
        assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
        ps.opt_head_norm_backward(x, x, w, y, dq_weight=torch.empty(dim, device="cuda"))
        ps.opt_head_norm_backward(tail, tail, w, y1)
        assert torch.equal(y[-5:], y1) and (y[:-5] == 0).all()
    del y
    ct, st = ps.e4m3_storage(cols, rows)
    ps.opt_dequantize(c, s, codes_t=ct, scales_t=st)
    last = (rows - 5) // 128 * 128
    piece = storage(cols, rows - last)
    ps.opt_quantize(x[last:].contiguous().new_zeros(rows - last, cols).copy_(torch.nn.functional.pad(
        torch.from_numpy(ref.values(c1, s1)).to(torch.bfloat16).cuda(), (0, 0, rows - last - 5, 0))), codes_t=piece[0], scales_t=piece[1])
    assert torch.equal(ct[:, last:], piece[0])


def run_all(stream=None, workspace=True):
    """Each operator once on a stream; its outputs."""
    x, u, dy = (matrix(300, 769, "bf16", 100 + i) for i in range(3))
    q, dq_out = matrix(300, 512, "bf16", 103), matrix(300, 512, "bf16", 104)
    w = torch.ones(64, device="cuda")
    cos, sin = tables(300, 64)
    gk, uk, yk, t, qk = (storage(*n) for n in ((300, 769), (300, 769), (300, 769), (769, 300), (300, 512)))
    y, dg, du, q_out, dq, dw = (torch.empty_like(v) for v in (x, x, x, q, q, w))
    torch.cuda.synchronize()
    ps.opt_gated(x, u, y=y, codes=yk[0], scales=yk[1], gate_kept=gk, up_kept=uk, stream=stream)
    ps.opt_gated_backward(dy, gk, uk, dgate=dg, dup=du, y_codes_t=t, stream=stream)
    ps.opt_dequantize(*gk, x=y, stream=stream)
    ps.opt_head_norm(q, w, q_out, cos=cos, sin=sin, q_kept=qk, stream=stream)
    ps.opt_head_norm_backward(dq_out, qk, w, dq, dq_weight=dw, cos=cos, sin=sin, stream=stream)
    torch.cuda.synchronize()
    return [y, dg, du, *t, *gk, *yk, q_out, dq, dw]


def test_repeats_and_streams_bit_for_bit():
    first = run_all()
    side = torch.cuda.Stream()
    for other in (run_all(), run_all(side), run_all(side.cuda_stream)):
        assert all(torch.equal(p, q) for p, q in zip(first, other))


def test_a_block_between_products_replays_from_a_graph():
    """Forward and backward through head norm and gated activation in one graph, replayed
    on new inputs."""
    rows, dim = 200, 64
    x, u, dy = (matrix(rows, 384, "bf16", 110 + i) for i in range(3))
    w = torch.ones(dim, device="cuda")
    cos, sin = tables(rows, dim)
    work = torch.empty(ps.opt_head_norm_backward_workspace(rows, 6, 0, dim), dtype=torch.uint8, device="cuda")

    def outputs():
        return dict(q=torch.empty_like(x), dq=torch.empty_like(x), dw=torch.empty_like(w), qk=storage(rows, 384), gk=storage(rows, 384),
                    uk=storage(rows, 384), yk=storage(rows, 384), ct=storage(384, rows), dg=torch.empty_like(x), du=torch.empty_like(x))

    def calls(o):
        ps.opt_head_norm(x, w, o["q"], cos=cos, sin=sin, q_kept=o["qk"])
        ps.opt_gated(o["q"], u, codes=o["yk"][0], scales=o["yk"][1], gate_kept=o["gk"], up_kept=o["uk"])
        ps.opt_gated_backward(dy, o["gk"], o["uk"], dgate=o["dg"], dup=o["du"], y_codes_t=o["ct"])
        ps.opt_head_norm_backward(o["dg"], o["qk"], w, o["dq"], dq_weight=o["dw"], cos=cos, sin=sin, workspace=work)

    got, want = outputs(), outputs()
    calls(got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(got)
    x.mul_(1.5)
    u.mul_(-0.5)
    graph.replay()
    calls(want)
    torch.cuda.synchronize()
    for k, v in want.items():
        assert all(torch.equal(a, b) for a, b in zip(v, got[k])) if isinstance(v, tuple) else torch.equal(v, got[k])


# ------------------------------------- forms that large calls and others' sets of outputs take
def training_outputs(rows, cols):
    """Every operand that a training step asks for, and nothing plain."""
    return {**{n: storage(rows, cols) for n in ("dgate_codes", "dup_codes")},
            **{n: storage(cols, rows) for n in ("dgate_codes_t", "dup_codes_t", "y_codes_t")}}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 8), (128, 128), (130, 264), (257, 1032), (2000, 1400), (1, 14336), (3000, 24), (77, 4096)])
def test_all_operands_are_those_of_single_calls(kind, rows, cols):
    """The training step's set of outputs (BF16, kept inputs) has a kernel of its own: the same
    bits as from calls for one output each, with several tiles to a CTA, tiles that end inside,
    zero blocks, infinities and NaN."""
    g, u, dy = spread(rows, cols, "bf16", 120), matrix(rows, cols, "bf16", 121), matrix(rows, cols, "bf16", 122, std=1e-2)
    if rows > 100:
        g[5, 3], u[70, 1], dy[90, 2], dy[100, 9], g[40] = float("nan"), float("inf"), float("-inf"), float("nan"), 0.0
        dy[110:120] = 0.0
    gk, uk = kept(g), kept(u)
    out = training_outputs(rows, cols)
    ps.opt_gated_backward(dy, gk, uk, activation=kind, **out)
    for name, got in out.items():
        want = storage(*got[0].shape)
        ps.opt_gated_backward(dy, gk, uk, activation=kind, **{name: want})
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), name
    if kind == "silu":
        plain = blank(rows, cols, "bf16"), blank(rows, cols, "bf16")
        more = training_outputs(rows, cols)
        ps.opt_gated_backward(dy, gk, uk, activation=kind, dgate=plain[0], dup=plain[1], **more)
        for name, got in out.items():
            assert torch.equal(got[0], more[name][0]) and torch.equal(got[1], more[name][1]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(9001, 264, 0), (3001, 2056, 8), (12000, 33, 0)])
def test_many_rows_are_those_of_fewer(dtype, rows, cols, pad):
    """More rows than the device takes at once: the same bits as slice by slice."""
    g, u, dy = spread(rows, cols, dtype, 130, pad), matrix(rows, cols, dtype, 131, pad), matrix(rows, cols, dtype, 132, pad)
    y, pair, gk, uk = blank(rows, cols, dtype), storage(rows, cols), storage(rows, cols), storage(rows, cols)
    dg, du = blank(rows, cols, dtype), blank(rows, cols, dtype)
    ps.opt_gated(g, u, y=y, codes=pair[0], scales=pair[1], gate_kept=gk, up_kept=uk)
    ps.opt_gated_backward(dy, gk, uk, dgate=dg, dup=du)
    tiles = ps.opt_scales_bytes(128, cols)
    for a in range(0, rows, 1280):                          # whole panels of scale tiles
        b = min(a + 1280, rows)
        part = lambda t: t[a:b]  # noqa: E731
        y1, p1, g1, u1 = blank(b - a, cols, dtype), storage(b - a, cols), storage(b - a, cols), storage(b - a, cols)
        ps.opt_gated(part(g), part(u), y=y1, codes=p1[0], scales=p1[1], gate_kept=g1, up_kept=u1)
        assert torch.equal(y1, part(y))
        for one, whole in ((p1, pair), (g1, gk), (u1, uk)):
            assert torch.equal(one[0], part(whole[0]))
            assert (ref.scale_bytes_of(one[1], b - a, cols) == ref.scale_bytes_of(whole[1][a // 128 * tiles:], b - a, cols)).all()
        d1, e1 = blank(b - a, cols, dtype), blank(b - a, cols, dtype)
        ps.opt_gated_backward(part(dy), g1, u1, dgate=d1, dup=e1)
        assert torch.equal(d1, part(dg)) and torch.equal(e1, part(du))


@pytest.mark.parametrize("rows,cols", [(3001, 4008), (20000, 130), (130, 20000)])
def test_many_tiles_turned(rows, cols):
    """More tiles than the device holds at once: the quantizer's codes of the same values."""
    pair = kept(matrix(rows, cols, "f32", 140, std=0.3))
    x, (ct, st), (c1, s1) = blank(rows, cols, "f32"), storage(cols, rows), storage(cols, rows)
    ps.opt_dequantize(*pair, x=x, codes_t=ct, scales_t=st)
    ps.opt_quantize(x, codes_t=c1, scales_t=s1)
    assert torch.equal(ct, c1) and torch.equal(st, s1)
    ps.opt_dequantize(*pair, codes_t=c1, scales_t=s1)
    assert torch.equal(ct, c1) and torch.equal(st, s1)
    y = blank(rows, cols, "bf16")
    ps.opt_dequantize(*pair, x=y)
    assert torch.equal(y, x.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq,hk,dim,rot,interleaved", [
    (9000, 9, 2, 64, 64, False), (6001, 12, 12, 128, 64, True), (4000, 1, 0, 256, 256, False), (5000, 40, 3, 16, 16, False),
    (9000, 5, 1, 96, 96, False), (7000, 3, 2, 100, 50, True), (3, 2000, 300, 128, 128, False), (2, 700, 0, 80, 16, True),
    (3000, 21, 2, 36, 36, False), (700, 19, 3, 250, 100, True), (2000, 13, 0, 63, 62, False), (1500, 9, 4, 80, 40, False)])
def test_many_heads_are_those_of_fewer(dtype, rows, hq, hk, dim, rot, interleaved):
    """More rows than warps, and more heads than a strip: the same bits as slice by slice, for
    kept and plain inputs; the weights' gradients in any case near the exact ones."""
    cos, sin = tables(500, rot)
    at = places(rows, 500, 3)
    how = dict(cos=cos, sin=sin, interleaved=interleaved)
    w = [(1 + 0.2 * matrix(1, dim, "f32", 150 + i)[0]).contiguous() for i in range(2)]
    x = [matrix(rows, h * dim, dtype, 152 + i) for i, h in enumerate((hq, hk))]
    d = [matrix(rows, h * dim, dtype, 154 + i, std=0.1) for i, h in enumerate((hq, hk))]

    def both(a, b, source):
        n = b - a
        out, keep = [blank(n, h * dim, dtype) for h in (hq, hk)], [storage(n, h * dim) for h in (hq, hk)]
        dx, dw = [blank(n, h * dim, dtype) for h in (hq, hk)], [torch.empty(dim, device="cuda") for _ in range(2)]
        t = [v[a:b] for v in x]
        k = dict(k=t[1], k_weight=w[1], k_out=out[1], k_kept=keep[1]) if hk else {}
        ps.opt_head_norm(t[0], w[0], out[0], q_kept=keep[0], positions=at[a:b], **k, **how)
        s = keep if source == "kept" else t
        k = dict(dk_out=d[1][a:b], k=s[1], k_weight=w[1], dk=dx[1], dk_weight=dw[1]) if hk else {}
        ps.opt_head_norm_backward(d[0][a:b], s[0], w[0], dx[0], dq_weight=dw[0], positions=at[a:b], **k, **how)
        return out, [p[0] for p in keep], dx, dw

    step = max(rows // 7, 1)
    for source in ("plain", "kept"):
        out, codes, dx, dw = both(0, rows, source)
        for a in range(0, rows, step):
            b = min(a + step, rows)
            for whole, part in zip((out, codes, dx), both(a, b, source)):
                assert all(torch.equal(p, q[a:b]) for p, q in zip(part, whole))
        if source == "plain":
            c, s = (t.double().cpu().numpy()[at.cpu().numpy()] for t in (cos, sin))
            for i, h in enumerate((hq, hk)[:2 if hk else 1]):
                _, _, want, size = act.head_norm_backward(f64(heads_of(d[i], dim)), f64(heads_of(x[i], dim)), f64(w[i]), 1e-5, c, s, rot, interleaved)
                assert (np.abs(f64(dw[i]) - want) <= E24 * (rows * h + dim / 32 + 30) * size).all()


def test_rows_far_apart():
    """Rows so far apart that 32-bit offsets inside a tile would not hold them."""
    pitch, rows, cols = (1 << 24) + 64, 5, 264
    wide = [torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda").view(rows, pitch)[:, :cols] for _ in range(3)]
    near = [matrix(rows, cols, "bf16", 160 + i) for i in range(3)]
    for a, b in zip(wide, near):
        a.copy_(b)
    got, want = training_outputs(rows, cols), training_outputs(rows, cols)
    ps.opt_gated_backward(wide[0], wide[1], wide[2], **got)
    ps.opt_gated_backward(near[0], near[1], near[2], **want)
    for name in got:
        assert all(torch.equal(p, q) for p, q in zip(got[name], want[name])), name
    codes = [torch.empty(rows * pitch, dtype=torch.uint8, device="cuda").view(rows, pitch)[:, :cols] for _ in range(2)]
    kg, ku = kept(near[1]), kept(near[2])
    codes[0].copy_(kg[0])
    codes[1].copy_(ku[0])
    ps.opt_gated_backward(near[0], (codes[0], kg[1]), (codes[1], ku[1]), **got)
    ps.opt_gated_backward(near[0], kg, ku, **want)
    for name in got:
        assert all(torch.equal(p, q) for p, q in zip(got[name], want[name])), name
    a, b = storage(cols, rows), storage(cols, rows)
    ps.opt_dequantize(codes[0], kg[1], codes_t=a[0], scales_t=a[1])
    ps.opt_dequantize(*kg, codes_t=b[0], scales_t=b[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    w = torch.ones(8, device="cuda")
    one, two = torch.empty_like(near[0]), torch.empty_like(near[0])
    ps.opt_head_norm(wide[1], w, one)
    ps.opt_head_norm(near[1], w, two)
    assert torch.equal(one, two)
    ps.opt_head_norm_backward(wide[0], wide[1], w, one)
    ps.opt_head_norm_backward(near[0], near[1], w, two)
    assert torch.equal(one, two)


@pytest.mark.parametrize("rows,pitch", [(1100, (1 << 22) + 64), (300, (1 << 24) + 64)])
def test_offsets_past_32_bits(rows, pitch):
    """Matrices that are columns of rows so long that their last ones lie past 2^32 elements: the
    same bits as of matrices of their own, for inputs and outputs of every call."""
    cols = 264
    wide = torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda").view(rows, pitch)
    wide8 = torch.empty(max(rows, cols) * pitch, dtype=torch.uint8, device="cuda").view(max(rows, cols), pitch)
    places = iter(range(0, 1 << 20, 1152))      # columns of either

    def far(like):
        at = next(places)
        return wide[:, at:at + cols] if like is None else wide8[:like[0], at:at + like[1]]

    g, u, dy = (matrix(rows, cols, "bf16", 170 + i) for i in range(3))
    fg, fu, fd = far(None), far(None), far(None)
    for a, b in ((fg, g), (fu, u), (fd, dy)):
        a.copy_(b)

    def pair(r, c, away):
        codes, scales = storage(r, c)
        return (far((r, c)) if away else codes), scales

    def run(away, gate, up, d):
        new = lambda: far(None) if away else torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        y, yc, gk, uk = new(), pair(rows, cols, away), pair(rows, cols, away), pair(rows, cols, away)
        ps.opt_gated(gate, up, y=y, codes=yc[0], scales=yc[1], gate_kept=gk, up_kept=uk)
        every = {**{n: pair(rows, cols, away) for n in ("dgate_codes", "dup_codes")},
                 **{n: pair(cols, rows, away) for n in ("dgate_codes_t", "dup_codes_t", "y_codes_t")}}
        ps.opt_gated_backward(d, gk, uk, **every)
        dg, du, dgc, dgt = new(), new(), pair(rows, cols, away), pair(cols, rows, away)
        ps.opt_gated_backward(d, gate, up, dgate=dg, dup=du)
        ps.opt_gated_backward(d, gk, uk, dgate_codes=dgc)
        ps.opt_gated_backward(d, gate, up, dgate_codes_t=dgt)
        x, xt, xu = new(), pair(cols, rows, away), new()
        ps.opt_dequantize(*gk, x=x, codes_t=xt[0], scales_t=xt[1])
        ps.opt_dequantize(*gk, x=xu)
        out = [y, *yc, *gk, *uk, dg, du, *dgc, *dgt, x, *xt, xu] + [t for p in every.values() for t in p]
        for dim in (8, 24, 33, 264):                  # strips of either kind, single elements, long heads
            w = torch.ones(dim, device="cuda")
            n, dn, dk, dw = new(), new(), new(), torch.empty(dim, device="cuda")
            held = pair(rows, cols, away)
            ps.opt_head_norm(gate, w, n, q_kept=held)
            ps.opt_head_norm_backward(d, gate, w, dn, dq_weight=dw)
            ps.opt_head_norm_backward(d, held, w, dk)
            out += [n, *held, dn, dw, dk]
        return out

    assert (rows - 1) * pitch >= 1 << 32 and rows <= 1152
    for i, (a, b) in enumerate(zip(run(True, fg, fu, fd), run(False, g, u, dy))):
        assert torch.equal(a, b), i


def test_rows_behind_the_last_stay():
    """Codes and plain outputs of a padded batch: rows behind the given ones keep what they hold."""
    rows, cols, more = 200, 256, 56
    buffers = {n: torch.full((rows + more, cols), 0x55, dtype=torch.uint8, device="cuda") for n in ("codes", "gate", "up", "dgate", "dup")}
    tall = torch.full((rows + more, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    scales = lambda: torch.zeros(ps.opt_scales_bytes(rows, cols), dtype=torch.uint8, device="cuda")  # noqa: E731
    pair = {n: (b[:rows], scales()) for n, b in buffers.items()}
    x = matrix(rows, cols, "bf16", 170)
    ps.opt_gated(x, x, y=tall[:rows], codes=pair["codes"][0], scales=pair["codes"][1], gate_kept=pair["gate"], up_kept=pair["up"])
    t = {n: storage(cols, rows) for n in ("dgate_codes_t", "dup_codes_t", "y_codes_t")}
    ps.opt_gated_backward(x, pair["gate"], pair["up"], dgate_codes=pair["dgate"], dup_codes=pair["dup"], **t)
    ps.opt_dequantize(*pair["gate"], x=tall[:rows], codes_t=t["y_codes_t"][0], scales_t=t["y_codes_t"][1])
    ps.opt_head_norm(x, torch.ones(64, device="cuda"), tall[:rows])
    assert all((b[rows:] == 0x55).all() for b in buffers.values()) and (tall[rows:] == 7).all()


def test_two_graphs_and_a_call_at_once():
    """Two captured backward passes with workspaces of their own, replayed on two streams while
    eager calls run on a third: each has its own results."""
    rows, heads, dim = 3000, 6, 64
    w = torch.ones(dim, device="cuda")
    cos, sin = tables(rows, dim)
    jobs = []
    for i in range(3):
        x, d = matrix(rows, heads * dim, "bf16", 180 + i), matrix(rows, heads * dim, "bf16", 190 + i)
        jobs.append(dict(x=x, d=d, dx=torch.empty_like(x), dw=torch.empty(dim, device="cuda"),
                         work=torch.empty(ps.opt_head_norm_backward_workspace(rows, heads, 0, dim), dtype=torch.uint8, device="cuda")))

    def call(j, stream=None):
        ps.opt_head_norm_backward(j["d"], j["x"], w, j["dx"], dq_weight=j["dw"], cos=cos, sin=sin, workspace=j["work"], stream=stream)

    want = []
    for j in jobs:
        call(j)
        torch.cuda.synchronize()
        want.append((j["dx"].clone(), j["dw"].clone()))
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs = []
    for j, s in zip(jobs[:2], streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(j)
            call(j)
        graphs.append(g)
    for j in jobs:
        j["dx"].zero_()
        j["dw"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        call(jobs[2], streams[2])
    torch.cuda.synchronize()
    for j, (dx, dw) in zip(jobs, want):
        assert torch.equal(j["dx"], dx) and torch.equal(j["dw"], dw)


def test_refused_calls_write_nothing():
    x, y = matrix(4, 64, "bf16", 200), torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w, pair = torch.ones(64, device="cuda"), storage(4, 64)
    cos, sin = tables(4, 64)
    bad = [lambda: ps.opt_gated(x, x[:3], y=y), lambda: ps.opt_gated(x, y=y.float()), lambda: ps.opt_gated(x, y=y, gate_kept=(pair[0], pair[1][:256])),
           lambda: ps.opt_gated(x, y=y, up_kept=pair), lambda: ps.opt_gated(x), lambda: ps.opt_gated_backward(x, pair, x, dgate=y, dup=y),
           lambda: ps.opt_gated_backward(x, x, dgate=y, dup=y), lambda: ps.opt_gated_backward(x, x, x),
           lambda: ps.opt_gated_backward(x, x, x, dgate=y, dgate_codes_t=pair), lambda: ps.opt_dequantize(*pair),
           lambda: ps.opt_dequantize(*pair, x=y[:3]), lambda: ps.opt_head_norm(x, w[:63], y), lambda: ps.opt_head_norm(x, w, y, k=x),
           lambda: ps.opt_head_norm(x, w, y, k_out=y), lambda: ps.opt_head_norm(x, w, y, cos=cos), lambda: ps.opt_head_norm(x, w, y, cos=cos, sin=sin[:3]),
           lambda: ps.opt_head_norm(x, w, y, cos=cos, sin=sin, positions=torch.zeros(3, dtype=torch.int64, device="cuda")),
           lambda: ps.opt_head_norm(x, w, y, cos=cos, sin=sin, positions=torch.zeros(4, dtype=torch.int32, device="cuda")),
           lambda: ps.opt_head_norm(x, w, y, cos=cos.t(), sin=sin.t()), lambda: ps.opt_head_norm(x, w, y, eps=-1.0), lambda: ps.opt_head_norm(x, w, y, eps=1e300),
           lambda: ps.opt_head_norm(x, w, y, k=x[:3], k_weight=w, k_out=y[:3]), lambda: ps.opt_head_norm(x, w[:32], y, cos=cos, sin=sin),
           lambda: ps.opt_head_norm_backward(x, pair, w, y, dk_out=x, k=x, k_weight=w, dk=y), lambda: ps.opt_head_norm_backward(x, x, w, y, k=x),
           lambda: ps.opt_head_norm_backward(x, x, w, y, dq_weight=torch.empty(64, device="cuda"), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for call in bad:
        with pytest.raises((ValueError, ps.OptError)):
            call()
    torch.cuda.synchronize()
    assert (y == 7).all() and (pair[1] == 0xEE).all()
