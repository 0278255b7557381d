"""GPU tests of what the binding of the training-layer operators refuses before a
call, given CUDA tensors."""
import pytest
import torch

import precision_states_gb300 as ps

pytestmark = pytest.mark.gpu


def test_numbers_that_their_types_do_not_hold_are_refused():
    x = torch.ones(4, 8, device="cuda")
    w, rstd = torch.ones(8, device="cuda"), torch.ones(4, device="cuda")
    codes, scales = ps.e4m3_storage(4, 8)
    y = torch.full_like(x, 7.0)
    for bad in (dict(seed=-1), dict(seed=1 << 64), dict(tensor_index=-1), dict(tensor_index=1 << 32), dict(step=1 << 63), dict(p="0.1")):
        for call in (lambda **f: ps.opt_dropout(x, y, **{"p": 0.1, **f}), lambda **f: ps.opt_rms_norm(x, w, y=y, **f),
                     lambda **f: ps.opt_rms_norm_backward(x, x, w, rstd, y, **f)):
            with pytest.raises(ValueError):
                call(**bad)
    with pytest.raises(ValueError):
        ps.opt_rms_norm(x, w, eps=1e300, y=y)
    with pytest.raises(ValueError):
        ps.opt_quantize(x, codes, scales, block_rows=1 << 40)
    ps.opt_dropout(x, y.clone(), 0.1, seed=(1 << 64) - 1, tensor_index=(1 << 32) - 1, step=(1 << 63) - 1)
    assert (y == 7).all()


def test_workspace_of_another_place_or_layout_is_refused():
    x = torch.ones(600, 8, device="cuda")
    w, rstd, dw = torch.ones(8, device="cuda"), torch.ones(600, device="cuda"), torch.full((8,), 7.0, device="cuda")
    need = ps.opt_rms_norm_backward_workspace(600, 8)
    assert need == 600 * 32
    strided = torch.empty(need, 2, dtype=torch.uint8, device="cuda")[:, 0]
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.uint8).view(600, 32), strided):
        with pytest.raises(ValueError):
            ps.opt_rms_norm_backward(x, x, w, rstd, torch.empty_like(x), dweight=dw, workspace=bad)
    with pytest.raises(ps.OptError) as e:
        ps.opt_rms_norm_backward(x, x, w, rstd, torch.empty_like(x), dweight=dw,
                                 workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ps.OPT_EINVAL and (dw == 7).all()
