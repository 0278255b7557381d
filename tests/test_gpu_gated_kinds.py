"""GPU tests of the gated activation and its gradients against the definitions in float64,
every activation with and without `up`, in whole chunks and in rows that begin anywhere, by
each set of inputs kept and of outputs that has a kernel of its own."""
import numpy as np
import pytest
import torch

import activation_reference as act
import precision_states_gb300 as ps
from test_gpu_activations import KINDS, as_values, kept, spread, storage, within
from test_gpu_layer import blank, f64, matrix

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
# rows, columns, padding, shift: whole chunks (whole tiles, and tiles that end inside), and any place
PLACES = [(256, 512, 0, 0), (131, 1032, 8, 0), (130, 517, 3, 1)]


def values32(x):
    return x.float().cpu().numpy()


@pytest.mark.parametrize("rows,cols,pad,shift", PLACES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("has_up", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_forward(kind, has_up, dtype, rows, cols, pad, shift):
    """To y and to codes, with every set of the inputs kept."""
    g, u = spread(rows, cols, dtype, 41, pad, shift), matrix(rows, cols, dtype, 42, pad) if has_up else None
    f, _, d, _ = act.activation(f64(g), kind)
    uv = f64(u) if has_up else 1.0
    want, d = f * uv, d * np.abs(uv) + E24 * np.abs(f * uv)
    y = blank(rows, cols, dtype)
    ps.opt_gated(g, u, activation=kind, y=y)
    within(y, want, dtype, d)
    for keep_gate, keep_up in ((False, False), (True, False), (False, True), (True, True)):
        if keep_up and not has_up:
            continue
        for plain in (False, True):
            pair, gk, uk, y2 = storage(rows, cols), storage(rows, cols), storage(rows, cols), blank(rows, cols, dtype)
            ps.opt_gated(g, u, activation=kind, y=y2 if plain else None, codes=pair[0], scales=pair[1],
                         gate_kept=gk if keep_gate else None, up_kept=uk if keep_up else None)
            act.check_codes(*pair, want, d)
            assert act.untouched(pair[1], rows, cols, 0xEE)
            if plain:
                assert (y2 == y).all()
            for on, k, x in ((keep_gate, gk, g), (keep_up, uk, u)):
                if on:
                    act.check_kept(*k, values32(x))
                    assert act.untouched(k[1], rows, cols, 0xEE)


OUTPUTS = {
    "all five": ["dgate_codes", "dgate_codes_t", "dup_codes", "dup_codes_t", "y_codes_t"],
    "without y": ["dgate_codes", "dgate_codes_t", "dup_codes", "dup_codes_t"],
    "by columns": ["dgate_codes_t", "dup_codes_t", "y_codes_t"],
    "by rows": ["dgate_codes", "dup_codes"],
    "plain": ["dgate", "dup"],
    "plain and by columns": ["dgate", "dup", "dgate_codes_t", "dup_codes_t", "y_codes_t"],
}


@pytest.mark.parametrize("outputs", list(OUTPUTS))
@pytest.mark.parametrize("rows,cols,pad,shift", PLACES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("source", ["plain", "kept"])
@pytest.mark.parametrize("has_up", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_backward(kind, has_up, source, dtype, rows, cols, pad, shift, outputs):
    g, u = spread(rows, cols, dtype, 43, pad, shift), matrix(rows, cols, dtype, 44, pad) if has_up else None
    dy = matrix(rows, cols, dtype, 45, pad, shift, std=1e-2)
    if source == "kept":
        g, u = kept(g), kept(u) if has_up else None
    gv, uv, dv = as_values(g), as_values(u) if has_up else 1.0, f64(dy)
    f, df, d, dd = act.activation(gv, kind)
    want = {"dgate": dv * df * uv, "dup": dv * f, "y": f * uv}
    off = {"dgate": np.abs(dv * uv) * dd + 3 * E24 * np.abs(want["dgate"]), "dup": np.abs(dv) * d + 2 * E24 * np.abs(want["dup"]),
           "y": np.abs(uv) * d + 2 * E24 * np.abs(want["y"])}
    names = [n for n in OUTPUTS[outputs] if has_up or not n.startswith("dup")]
    out = {n: storage(cols, rows) if n.endswith("_t") else storage(rows, cols) if n.endswith("_codes") else blank(rows, cols, dtype, pad)
           for n in names}
    ps.opt_gated_backward(dy, g, u, activation=kind, **out)
    for n, got in out.items():
        of = n.split("_")[0]
        if n.endswith("_t"):
            act.check_codes(*got, want[of].T, off[of].T)
            assert act.untouched(got[1], cols, rows, 0xEE)
        elif n.endswith("_codes"):
            act.check_codes(*got, want[of], off[of])
            assert act.untouched(got[1], rows, cols, 0xEE)
        else:
            within(got, want[of], dtype, off[of])


@pytest.mark.parametrize("rows,cols,pad,shift", PLACES)
@pytest.mark.parametrize("source", ["plain", "kept"])
@pytest.mark.parametrize("kind", KINDS)
def test_codes_are_the_quantizers_of_the_fp32_values(kind, source, rows, cols, pad, shift):
    """Of fp32 matrices codes and plain outputs are rounded from the same values: the codes are
    those that opt_quantize makes of the plain ones, bit for bit, with infinities and NaN, zero
    blocks, and blocks whose values leave fp32 or are subnormal."""
    g, u, dy = spread(rows, cols, "f32", 46, pad, shift), matrix(rows, cols, "f32", 47, pad), matrix(rows, cols, "f32", 48, pad, shift, std=1e-2)
    dy[3], u[7], dy[:, 9] = 0.0, 0.0, 0.0
    dy[11, 5], u[11, 200], dy[90, 2] = float("nan"), float("inf"), float("-inf")
    dy[20:24] *= 1e38
    u[30:34] *= 3e37
    dy[40:44] *= 1e-37
    if source == "kept":
        g, u = kept(g), kept(u)
    plain = {n: blank(rows, cols, "f32", pad) for n in ("dgate", "dup")}
    coded = {n + "_codes": storage(rows, cols) for n in ("dgate", "dup")}
    turned = {n + "_codes_t": storage(cols, rows) for n in ("dgate", "dup")}
    ps.opt_gated_backward(dy, g, u, activation=kind, **plain, **coded, **turned)
    by_rows = {n + "_codes": storage(rows, cols) for n in ("dgate", "dup")}
    ps.opt_gated_backward(dy, g, u, activation=kind, **by_rows)
    for n in ("dgate", "dup"):
        c, t = storage(rows, cols), storage(cols, rows)
        ps.opt_quantize(plain[n], *c, *t)
        assert not plain[n].isfinite().all()
        for got, want in ((coded[n + "_codes"], c), (by_rows[n + "_codes"], c), (turned[n + "_codes_t"], t)):
            odd = (want[0] & 0x7F) == 0x7F            # a NaN's sign is not looked at
            assert torch.equal((got[0] & 0x7F) == 0x7F, odd) and torch.equal(got[0][~odd], want[0][~odd]) and torch.equal(got[1], want[1])
