"""CPU tests of the C ABI of the gated activation, the heads' norm with rotation,
their gradients and kept activations: the packed arguments have the header's layout,
workspace sizes, and every refusal, which the library makes on the host before any
launch."""
import os
import re

import pytest
import torch

import precision_states_gb300 as ps
from conftest import ROOT
from precision_states_gb300 import layer

P = 0x10000          # a 16-byte aligned address that no refused call looks at
BIG = 1 << 31


def call(name, **fields):
    return getattr(ps.lib(), name)(bytes(getattr(layer, name + "_args")(**fields)), None)


@pytest.mark.parametrize("name", ["opt_dequantize", "opt_gated", "opt_gated_backward", "opt_head_norm", "opt_head_norm_backward"])
def test_packed_arguments_are_the_struct(name):
    st = getattr(layer, name + "_args")
    vals = list(range(1, len(st._fields_) + 1))
    assert layer.packer(st)(*vals) == bytes(st(*vals))
    src = open(os.path.join(ROOT, "include", "opt_layer.h")).read()
    body = re.sub(r"/\*.*?\*/", "", re.search(r"typedef struct %s_args \{(.*?)\}" % name, src, re.S).group(1), flags=re.S)
    fields = [f.strip(" *\n") for line in body.split(";") for f in
              re.sub(r"^\s*(const\s+)?\w+\s*", "", line.strip()).split(",") if f.strip()]
    assert fields == [n for n, _ in st._fields_]
    assert ps.lib()[name](None, None) == ps.OPT_EINVAL


def test_header_constants():
    src = open(os.path.join(ROOT, "include", "opt_layer.h")).read()
    found = dict(re.findall(r"#define (OPT_[A-Z_]+)\s+(\d+)\n", src))
    assert {k: int(found["OPT_ACT_" + k.upper()]) for k in layer.ACTIVATIONS} == layer.ACTIVATIONS
    assert int(found["OPT_HEADS_INTERLEAVED"]) == ps.OPT_HEADS_INTERLEAVED


def test_head_workspace():
    for rows, hq, hk, dim, parts in ((0, 4, 2, 64, 0), (1, 32, 8, 128, 40), (4096, 32, 8, 128, 1024), (300, 1, 0, 33, 300), (5, 0, 0, 8, 0)):
        assert ps.opt_head_norm_backward_workspace(rows, hq, hk, dim) == parts * 2 * dim * 4
    ask = ps.lib().opt_head_norm_backward_workspace
    assert ask(-1, 1, 1, 64) == ps.OPT_EINVAL and ask(1, 1, 1, 0) == ps.OPT_EINVAL and ask(1, 1, 1, 1025) == ps.OPT_ELIMIT
    assert ask(1, 1 << 30, 1, 64) == ps.OPT_ELIMIT


DEQ = dict(d_codes=P, d_scales=P, d_x=P, codes_pitch=16, x_pitch=8, rows=2, cols=8, dtype=ps.OPT_BF16)
GATED = dict(d_gate=P, d_up=P, d_y=P, gate_pitch=8, up_pitch=8, y_pitch=8, rows=2, cols=8, dtype=ps.OPT_BF16, activation=0)
GRAD = dict(d_dy=P, d_gate=P, d_up=P, d_dgate=P, d_dup=P, dy_pitch=8, gate_pitch=8, up_pitch=8, dgate_pitch=8, dup_pitch=8, rows=2,
            cols=8, dtype=ps.OPT_F32, activation=3)
KEPT = dict(GRAD, d_gate_scales=P, d_up_scales=P, gate_pitch=16, up_pitch=16)
HEAD = dict(d_q=P, d_q_weight=P, d_q_out=P, d_k=P, d_k_weight=P, d_k_out=P, d_cos=P, d_sin=P, d_positions=P, q_pitch=64, q_out_pitch=64,
            k_pitch=32, k_out_pitch=32, rows=3, q_heads=2, k_heads=1, dim=32, rot=16, positions=9, dtype=ps.OPT_BF16,
            weight_dtype=ps.OPT_F32, eps=1e-5)
BACK = dict(d_dq_out=P, d_q=P, d_q_weight=P, d_dq=P, d_dq_weight=P, d_dk_out=P, d_k=P, d_k_weight=P, d_dk=P, d_dk_weight=P, d_cos=P,
            d_sin=P, d_positions=P, d_workspace=P, dq_out_pitch=64, q_pitch=64, dq_pitch=64, dk_out_pitch=32, k_pitch=32, dk_pitch=32,
            workspace_bytes=1 << 20, rows=3, q_heads=2, k_heads=1, dim=32, rot=16, positions=9, dtype=ps.OPT_BF16,
            weight_dtype=ps.OPT_F32, eps=1e-5)
E, U, A, L, OK = ps.OPT_EINVAL, ps.OPT_EUNSUPPORTED, ps.OPT_EALIGN, ps.OPT_ELIMIT, ps.OPT_OK


@pytest.mark.parametrize("name,base,change,status", [
    ("opt_dequantize", DEQ, dict(d_codes=0), E), ("opt_dequantize", DEQ, dict(d_scales=0), E), ("opt_dequantize", DEQ, dict(d_x=0), E),
    ("opt_dequantize", DEQ, dict(codes_pitch=24), A), ("opt_dequantize", DEQ, dict(d_codes=P + 8), A), ("opt_dequantize", DEQ, dict(x_pitch=7), E),
    ("opt_dequantize", DEQ, dict(d_codes_t=P, codes_t_pitch=16), E), ("opt_dequantize", DEQ, dict(d_codes_t=P, d_scales_t=P, codes_t_pitch=1), E),
    ("opt_dequantize", DEQ, dict(d_codes_t=P, d_scales_t=P, codes_t_pitch=8), A), ("opt_dequantize", DEQ, dict(d_x=P + 1), A),
    ("opt_dequantize", DEQ, dict(dtype=ps.OPT_E4M3), U), ("opt_dequantize", DEQ, dict(rows=-1), E), ("opt_dequantize", DEQ, dict(cols=BIG), L),
    ("opt_dequantize", DEQ, dict(reserved=1), E), ("opt_dequantize", DEQ, dict(rows=0, d_codes=0), OK),
    ("opt_gated", GATED, dict(d_gate=0), E), ("opt_gated", GATED, dict(d_y=0), E), ("opt_gated", GATED, dict(activation=4), E),
    ("opt_gated", GATED, dict(activation=-1), E), ("opt_gated", GATED, dict(dtype=ps.OPT_E2M2), U), ("opt_gated", GATED, dict(up_pitch=7), E),
    ("opt_gated", GATED, dict(d_up=P + 1), A), ("opt_gated", GATED, dict(d_codes=P, codes_pitch=16), E),
    ("opt_gated", GATED, dict(d_scales=P, codes_pitch=16), E), ("opt_gated", GATED, dict(d_gate_codes=P, d_gate_scales=P, gate_codes_pitch=8), A),
    ("opt_gated", GATED, dict(d_up=0, d_up_codes=P, d_up_scales=P, up_codes_pitch=16), E), ("opt_gated", GATED, dict(rows=BIG), L),
    ("opt_gated", GATED, dict(cols=0, d_gate=0), OK),
    ("opt_gated_backward", GRAD, dict(d_dy=0), E), ("opt_gated_backward", GRAD, dict(d_gate=0), E), ("opt_gated_backward", GRAD, dict(d_up=0), E),
    ("opt_gated_backward", GRAD, dict(d_dgate=0, d_dup=0), E), ("opt_gated_backward", GRAD, dict(d_up_scales=P), E),
    ("opt_gated_backward", GRAD, dict(dgate_pitch=7), E), ("opt_gated_backward", GRAD, dict(d_dup=P + 2), A),
    ("opt_gated_backward", GRAD, dict(d_dgate_codes=P, dgate_codes_pitch=16), E),
    ("opt_gated_backward", GRAD, dict(d_y_codes_t=P, d_y_scales_t=P, y_codes_t_pitch=1), E),
    ("opt_gated_backward", GRAD, dict(d_dup_codes_t=P, d_dup_scales_t=P + 4, dup_codes_t_pitch=16), A),
    ("opt_gated_backward", GRAD, dict(activation=9), E), ("opt_gated_backward", GRAD, dict(dtype=5), U), ("opt_gated_backward", GRAD, dict(cols=-1), E),
    ("opt_gated_backward", KEPT, dict(gate_pitch=24), A), ("opt_gated_backward", KEPT, dict(d_up_scales=0), E),
    ("opt_gated_backward", KEPT, dict(d_gate=P + 8), A), ("opt_gated_backward", KEPT, dict(rows=0, d_dy=0), OK),
    ("opt_head_norm", HEAD, dict(d_q=0), E), ("opt_head_norm", HEAD, dict(d_q_weight=0), E), ("opt_head_norm", HEAD, dict(d_k_out=0), E),
    ("opt_head_norm", HEAD, dict(q_pitch=63), E), ("opt_head_norm", HEAD, dict(dim=0), E), ("opt_head_norm", HEAD, dict(dim=2048, rot=16), L),
    ("opt_head_norm", HEAD, dict(rot=15), E), ("opt_head_norm", HEAD, dict(rot=34), E), ("opt_head_norm", HEAD, dict(rot=-2), E),
    ("opt_head_norm", HEAD, dict(flags=2), E), ("opt_head_norm", HEAD, dict(eps=-1.0), E), ("opt_head_norm", HEAD, dict(eps=float("inf")), E),
    ("opt_head_norm", HEAD, dict(d_cos=0), E), ("opt_head_norm", HEAD, dict(d_sin=P + 2), A), ("opt_head_norm", HEAD, dict(d_positions=P + 4), A),
    ("opt_head_norm", HEAD, dict(d_positions=0, positions=2), E), ("opt_head_norm", HEAD, dict(positions=-1), E),
    ("opt_head_norm", HEAD, dict(d_q_codes=P, q_codes_pitch=64), E), ("opt_head_norm", HEAD, dict(d_k_codes=P, d_k_scales=P, k_codes_pitch=33), A),
    ("opt_head_norm", HEAD, dict(q_heads=-1), E), ("opt_head_norm", HEAD, dict(q_heads=1 << 30), L), ("opt_head_norm", HEAD, dict(dtype=ps.OPT_E4M3), U),
    ("opt_head_norm", HEAD, dict(weight_dtype=7), U), ("opt_head_norm", HEAD, dict(d_q=P + 1), A), ("opt_head_norm", HEAD, dict(rows=0, d_q=0), OK),
    ("opt_head_norm", HEAD, dict(q_heads=0, k_heads=0, d_q=0), OK),
    ("opt_head_norm_backward", BACK, dict(d_workspace=0), E), ("opt_head_norm_backward", BACK, dict(workspace_bytes=9 * 256 - 1), E),
    ("opt_head_norm_backward", BACK, dict(d_workspace=P + 8), A), ("opt_head_norm_backward", BACK, dict(d_q_scales=P), E),
    ("opt_head_norm_backward", BACK, dict(d_k_scales=P), E), ("opt_head_norm_backward", BACK, dict(d_q_scales=P, d_k_scales=P, q_pitch=40), E),
    ("opt_head_norm_backward", BACK, dict(d_q_scales=P, d_k_scales=P, k_pitch=40), A), ("opt_head_norm_backward", BACK, dict(d_dq=0), E),
    ("opt_head_norm_backward", BACK, dict(d_dk_out=0), E), ("opt_head_norm_backward", BACK, dict(d_dq_weight=P + 2), A),
    ("opt_head_norm_backward", BACK, dict(flags=4), E), ("opt_head_norm_backward", BACK, dict(d_positions=0, positions=2), E),
    ("opt_head_norm_backward", BACK, dict(rows=-1), E), ("opt_head_norm_backward", BACK, dict(q_heads=0, k_heads=0, d_dq_weight=0, d_dk_weight=0), OK),
])
def test_refusals(name, base, change, status):
    assert call(name, **{**base, **change}) == status


def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros(4, 8), torch.ones(4)
    for refused in (lambda: ps.opt_gated(x, activation="silu", y=x), lambda: ps.opt_gated_backward(x, x, dgate=x),      # not on the device
                    lambda: ps.opt_dequantize(x, x, x=x), lambda: ps.opt_head_norm(x, w, x), lambda: ps.opt_head_norm_backward(x, x, w, x),
                    lambda: ps.opt_gated(x, activation="tanh", y=x)):
        with pytest.raises(ValueError):
            refused()
    for refused in (lambda: ps.opt_gated(x.double(), y=x), lambda: ps.opt_gated_backward(x.half(), x), lambda: ps.opt_head_norm(x.double(), w, x),
                    lambda: ps.opt_head_norm(x, w.half(), x)):
        with pytest.raises(ps.OptError) as e:
            refused()
        assert e.value.status == ps.OPT_EUNSUPPORTED
    assert layer._heads(torch.zeros(6, 32), "x", 8) == (6, 4, 32) and layer._heads(torch.zeros(6, 40)[:, :32], "x", 8) == (6, 4, 40)
    assert layer._heads(torch.zeros(6, 4, 8), "x", 8) == (6, 4, 32) and layer._heads(torch.zeros(6, 5, 8)[:, 1:], "x", 8) == (6, 4, 40)
    assert layer._heads(torch.zeros(2, 3, 4, 8), "x", 8) == (6, 4, 32)
    for bad in (torch.zeros(6, 33), torch.zeros(6, 4, 9), torch.zeros(6, 4, 16)[..., ::2], torch.zeros(4, 6, 8).transpose(0, 1)[:, ::2],
                torch.zeros(2, 4, 3, 8).transpose(1, 2), torch.zeros(8)):
        with pytest.raises(ValueError):
            layer._heads(bad, "x", 8)
    r = type("R", (), dict(f32=torch.float32, int64=torch.int64))
    for cos, sin, at in ((x, None, None), (None, x, None), (None, None, torch.zeros(4)), (x, x[:3], None), (x[0], x[0], None),
                         (x.half(), x.half(), None), (x, x, torch.zeros(4, dtype=torch.int32)), (x, x, torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            layer._turn(cos, sin, at, 4, -1, r)
    for pair in (x, (x,), (x, x, x)):
        with pytest.raises(ValueError):
            layer._pair(pair, "kept", 4, 8, -1, r)
