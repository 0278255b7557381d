"""CPU tests of the training-layer operators' C ABI: the header and the binding
agree, the packed arguments have the structs' layout, sizes of scale tiles, and
every refusal, which the library makes on the host before any launch."""
import ctypes
import os
import re

import pytest
import torch

import precision_states_gb300 as ps
from conftest import ROOT
from precision_states_gb300 import layer

P = 0x10000          # a 16-byte aligned address that no refused call looks at


def call(name, struct, **fields):
    a = struct(**fields)
    return getattr(ps.lib(), name)(bytes(a), None)


def test_header_binding_and_exports_agree():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "opt_layer.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(opt_[a-z0-9_]+)\s*\(", src)))
    assert names == sorted(layer.SIGS)
    for name in names:
        assert hasattr(ps.lib(), name) and hasattr(ps, name)


@pytest.mark.parametrize("name", ["opt_dropout", "opt_rms_norm", "opt_rms_norm_backward", "opt_quantize", "opt_matmul"])
def test_packed_arguments_are_the_struct(name):
    st = getattr(layer, name + "_args")
    vals = list(range(1, len(st._fields_) + 1))
    assert layer.packer(st)(*vals) == bytes(st(*vals))
    # the header's fields in the header's order
    src = open(os.path.join(ROOT, "include", "opt_layer.h")).read()
    body = re.sub(r"/\*.*?\*/", "", re.search(r"typedef struct %s_args \{(.*?)\}" % name, src, re.S).group(1), flags=re.S)
    fields = [f.strip(" *\n") for line in body.split(";") for f in
              re.sub(r"^\s*(const\s+)?\w+\s*", "", line.strip()).split(",") if f.strip()]
    assert fields == [n for n, _ in st._fields_]
    assert ps.lib()[name](None, None) == ps.OPT_EINVAL


def test_scales_bytes():
    for rows, cols, want in ((0, 0, 0), (1, 1, 512), (128, 512, 512), (129, 513, 2048), (4096, 4096, 32 * 8 * 512)):
        assert ps.opt_scales_bytes(rows, cols) == layer.scales_bytes(rows, cols) == want
    assert ps.lib().opt_scales_bytes(-1, 4) == ps.OPT_EINVAL
    assert ps.lib().opt_scales_bytes(1 << 31, 4) == ps.OPT_ELIMIT


def test_backward_workspace():
    for rows, cols in ((0, 7), (1, 1), (5, 769), (512, 4096)):             # few rows need none
        assert ps.opt_rms_norm_backward_workspace(rows, cols) == 0
    for rows, cols in ((513, 1), (512, 4097), (4096, 4095), (1, (1 << 21) + 1)):
        assert ps.opt_rms_norm_backward_workspace(rows, cols) == min(rows, 1024) * (-(-cols // 4) * 4) * 4
    assert ps.lib().opt_rms_norm_backward_workspace(-1, 4) == ps.OPT_EINVAL


DROPOUT = dict(d_x=P, d_y=P, x_pitch=8, y_pitch=8, rows=2, cols=8, p=0.1, dtype=ps.OPT_BF16)
NORM = dict(d_x=P, d_weight=P, d_y=P, x_pitch=8, y_pitch=8, rows=2, cols=8, dtype=ps.OPT_BF16, weight_dtype=ps.OPT_F32,
            eps=1e-5)
BACK = dict(d_dy=P, d_h=P, d_weight=P, d_rstd=P, d_dh=P, d_dweight=P, d_workspace=P, workspace_bytes=1 << 20, dy_pitch=8,
            h_pitch=8, dh_pitch=8, rows=600, cols=8, dtype=ps.OPT_F32, weight_dtype=ps.OPT_F32)
QUANT = dict(d_x=P, d_codes=P, d_scales=P, x_pitch=8, codes_pitch=16, rows=2, cols=8, dtype=ps.OPT_F32, block_rows=1)
MATMUL = dict(d_a=P, d_a_scales=P, d_b=P, d_b_scales=P, d_out=P, a_pitch=16, b_pitch=16, out_pitch=4, m=2, n=4, k=16,
              out_dtype=ps.OPT_F32)
BIG = 1 << 31


@pytest.mark.parametrize("name,base,change,status", [
    ("opt_dropout", DROPOUT, dict(p=1.5), ps.OPT_EINVAL), ("opt_dropout", DROPOUT, dict(p=-0.1), ps.OPT_EINVAL),
    ("opt_dropout", DROPOUT, dict(p=float("nan")), ps.OPT_EINVAL), ("opt_dropout", DROPOUT, dict(step=-1), ps.OPT_EINVAL),
    ("opt_dropout", DROPOUT, dict(d_x=0), ps.OPT_EINVAL), ("opt_dropout", DROPOUT, dict(d_y=0), ps.OPT_EINVAL),
    ("opt_dropout", DROPOUT, dict(x_pitch=7), ps.OPT_EINVAL), ("opt_dropout", DROPOUT, dict(rows=-1), ps.OPT_EINVAL),
    ("opt_dropout", DROPOUT, dict(cols=BIG), ps.OPT_ELIMIT), ("opt_dropout", DROPOUT, dict(dtype=ps.OPT_E4M3), ps.OPT_EUNSUPPORTED),
    ("opt_dropout", DROPOUT, dict(d_x=P + 1), ps.OPT_EALIGN), ("opt_dropout", DROPOUT, dict(d_residual=P, residual_pitch=2), ps.OPT_EINVAL),
    ("opt_dropout", DROPOUT, dict(rows=0, d_x=0), ps.OPT_OK), ("opt_dropout", DROPOUT, dict(cols=0, d_y=0), ps.OPT_OK),
    ("opt_rms_norm", NORM, dict(d_y=0), ps.OPT_EINVAL), ("opt_rms_norm", NORM, dict(d_weight=0), ps.OPT_EINVAL),
    ("opt_rms_norm", NORM, dict(eps=-1.0), ps.OPT_EINVAL), ("opt_rms_norm", NORM, dict(eps=float("nan")), ps.OPT_EINVAL),
    ("opt_rms_norm", NORM, dict(d_codes=P, codes_pitch=16), ps.OPT_EINVAL),
    ("opt_rms_norm", NORM, dict(d_codes=P, d_scales=P, codes_pitch=8), ps.OPT_EALIGN),
    ("opt_rms_norm", NORM, dict(d_codes=P + 8, d_scales=P, codes_pitch=16), ps.OPT_EALIGN),
    ("opt_rms_norm", NORM, dict(d_codes=P, d_scales=P + 4, codes_pitch=16), ps.OPT_EALIGN),
    ("opt_rms_norm", NORM, dict(weight_dtype=7), ps.OPT_EUNSUPPORTED), ("opt_rms_norm", NORM, dict(h_pitch=3, d_h=P), ps.OPT_EINVAL),
    ("opt_rms_norm", NORM, dict(d_rstd=P + 2), ps.OPT_EALIGN), ("opt_rms_norm", NORM, dict(p=2.0), ps.OPT_EINVAL),
    ("opt_rms_norm", NORM, dict(rows=0), ps.OPT_OK),
    ("opt_rms_norm_backward", BACK, dict(d_workspace=0), ps.OPT_EINVAL),
    ("opt_rms_norm_backward", BACK, dict(workspace_bytes=600 * 32 - 1), ps.OPT_EINVAL),
    ("opt_rms_norm_backward", BACK, dict(d_workspace=P + 4), ps.OPT_EALIGN),
    ("opt_rms_norm_backward", BACK, dict(d_rstd=0), ps.OPT_EINVAL), ("opt_rms_norm_backward", BACK, dict(d_dh=0), ps.OPT_EINVAL),
    ("opt_rms_norm_backward", BACK, dict(reserved=1), ps.OPT_EINVAL), ("opt_rms_norm_backward", BACK, dict(d_dx=P, dx_pitch=1), ps.OPT_EINVAL),
    ("opt_rms_norm_backward", BACK, dict(dtype=ps.OPT_E2M2), ps.OPT_EUNSUPPORTED), ("opt_rms_norm_backward", BACK, dict(cols=0), ps.OPT_OK),
    ("opt_quantize", QUANT, dict(block_rows=64), ps.OPT_EINVAL), ("opt_quantize", QUANT, dict(d_codes=0, d_scales=0), ps.OPT_EINVAL),
    ("opt_quantize", QUANT, dict(d_scales=0), ps.OPT_EINVAL), ("opt_quantize", QUANT, dict(codes_pitch=24), ps.OPT_EALIGN),
    ("opt_quantize", QUANT, dict(d_codes_t=P, d_scales_t=P, codes_t_pitch=1), ps.OPT_EINVAL),
    ("opt_quantize", QUANT, dict(d_x=P + 2), ps.OPT_EALIGN), ("opt_quantize", QUANT, dict(dtype=ps.OPT_E4M3), ps.OPT_EUNSUPPORTED),
    ("opt_quantize", QUANT, dict(rows=0), ps.OPT_OK),
    ("opt_matmul", MATMUL, dict(d_a=0), ps.OPT_EINVAL), ("opt_matmul", MATMUL, dict(d_b_scales=0), ps.OPT_EINVAL),
    ("opt_matmul", MATMUL, dict(a_pitch=17), ps.OPT_EALIGN), ("opt_matmul", MATMUL, dict(d_b=P + 8), ps.OPT_EALIGN),
    ("opt_matmul", MATMUL, dict(k=-1), ps.OPT_EINVAL), ("opt_matmul", MATMUL, dict(k=BIG), ps.OPT_ELIMIT),
    ("opt_matmul", MATMUL, dict(out_dtype=ps.OPT_E4M3), ps.OPT_EUNSUPPORTED), ("opt_matmul", MATMUL, dict(out_pitch=3), ps.OPT_EINVAL),
    ("opt_matmul", MATMUL, dict(d_addend=P, addend_pitch=3), ps.OPT_EINVAL), ("opt_matmul", MATMUL, dict(d_out=P + 2), ps.OPT_EALIGN),
    ("opt_matmul", MATMUL, dict(flags=2), ps.OPT_EINVAL),
    ("opt_matmul", MATMUL, dict(flags=ps.OPT_MATMUL_WAIT_DRILL), ps.OPT_EUNSUPPORTED),
    ("opt_matmul", MATMUL, dict(flags=ps.OPT_MATMUL_WAIT_DRILL, k=0), ps.OPT_EUNSUPPORTED), ("opt_matmul", MATMUL, dict(m=0, d_a=0), ps.OPT_OK),
])
def test_refusals(name, base, change, status):
    assert call(name, getattr(layer, name + "_args"), **{**base, **change}) == status


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ps.opt_dropout(x, x, 0.1)                              # not a CUDA tensor
    with pytest.raises(ps.OptError) as e:
        ps.opt_dropout(x.double(), x, 0.1)
    assert e.value.status == ps.OPT_EUNSUPPORTED
    with pytest.raises(ValueError):
        layer._matrix(torch.zeros(4, 8).t(), "x")
    with pytest.raises(ValueError):
        layer._matrix(torch.zeros(2, 4, 8).transpose(0, 1), "x")
    assert layer._matrix(torch.zeros(2, 3, 8), "x") == (6, 8, 8)
    assert layer._matrix(torch.zeros(3, 10)[:, :8], "x") == (3, 8, 10)
    assert layer._matrix(torch.zeros(8), "x") == (1, 8, 8)
    assert ctypes.sizeof(layer.opt_matmul_args) == 112


def test_matmul_form_without_tiles():
    """Answered on the host alone; refusals as in the product."""
    form = (ctypes.c_int32 * 5)(*[9] * 5)
    ask = lambda **f: ps.lib().opt_matmul_form(bytes(layer.opt_matmul_args(**f)), form)  # noqa: E731
    for size in (dict(m=8, n=4096, k=512), dict(m=4096, n=1, k=512), dict(m=300, n=300, k=0), dict(m=0, n=300, k=5)):
        assert ask(**size) == ps.OPT_OK and list(form) == [0] * 5
    assert ask(m=-1, n=4, k=4) == ps.OPT_EINVAL and ask(m=9, n=9, k=BIG) == ps.OPT_ELIMIT
    assert ps.lib().opt_matmul_form(None, form) == ps.OPT_EINVAL
    assert ps.lib().opt_matmul_form(bytes(layer.opt_matmul_args()), None) == ps.OPT_EINVAL
    assert ps.opt_matmul_form(torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(40, 64, dtype=torch.uint8)) == (0,) * 5
    with pytest.raises(ValueError):
        ps.opt_matmul_form(torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(40, 63, dtype=torch.uint8))


def test_given_workspace_is_looked_at():
    with pytest.raises(ValueError):
        layer._given_workspace(torch.zeros(64, dtype=torch.uint8), 0)          # not on the device
    assert layer._given_workspace(torch.zeros(4, 4), -1) == 64
    with pytest.raises(ValueError):
        layer._given_workspace(torch.zeros(4, 4).t()[:2], -1)
