"""GPU tests of the training-layer operators on a caller's stream while other
streams have work pending."""
import pytest
import torch

import precision_states_gb300 as ps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["stream", "pointer", "default"])
def test_norm_gradients_do_not_take_memory_that_pending_work_uses(form):
    """dweight's workspace (the call's own, over 512 rows) on a side stream, with a
    freed tensor of its size that pending work of the current stream still reads."""
    rows, cols = 2000, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.empty(rows, cols, device="cuda").normal_(generator=gen)
    dy = torch.empty(rows, cols, device="cuda").normal_(generator=gen)
    w, rstd = torch.ones(cols, device="cuda"), torch.rsqrt(h.square().mean(1) + 1e-5)
    dh, dw, want = torch.empty_like(h), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    need = ps.opt_rms_norm_backward_workspace(rows, cols)
    assert need > 0
    ps.opt_rms_norm_backward(dy, h, w, rstd, dh, dweight=want,
                             workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    here = torch.cuda.Stream() if form == "default" else torch.cuda.current_stream()
    stream = {"stream": side, "pointer": side.cuda_stream, "default": 0}[form]
    copy = torch.empty(need, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(here):
        for fill in (3, 5, 7):
            held = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            dw.zero_()
            torch.cuda.synchronize()
            torch.cuda._sleep(100_000_000)                  # about 50 ms
            copy.copy_(held)
            del held
            ps.opt_rms_norm_backward(dy, h, w, rstd, dh, dweight=dw, stream=stream)
            torch.cuda.synchronize()
            assert (copy == fill).all(), "another tensor's memory was written"
            assert torch.equal(dw, want)


def test_status_loses_no_flag_that_is_raised_while_it_is_asked():
    """Products whose waits run out on one stream, while another asks all the time."""
    codes, scales = ps.e4m3_storage(64, 256)
    out = torch.empty(64, 64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert ps.opt_layer_status() == 0
    for _ in range(200):
        ps.opt_matmul(codes, scales, codes, scales, out, stream=side, wait_drill=True)     # ends after 1 ms
        flags = 0
        while not side.query():
            flags |= ps.opt_layer_status()
        assert flags | ps.opt_layer_status() == ps.OPT_FLAG_WAIT_TIMEOUT
    assert ps.opt_layer_status() == 0
