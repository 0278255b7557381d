"""GPU tests of 8-bit operands of a single row, whose pitch is not looked at: whatever it
is, a call gives what it gives for the same operand in whole lines."""
import pytest
import torch

import layer_reference as ref
import precision_states_gb300 as ps
from test_gpu_layer import TD, blank, matrix

pytestmark = pytest.mark.gpu

# columns, and the pitch of the single row
ROWS = [(1, 1), (5, 5), (5, 1030), (16, 17), (129, 769), (513, 1030), (769, 769), (1030, 1030), (4096, 5001)]


def one_row(cols, pitch):
    """Codes of one row of the given pitch, and their scales."""
    codes = torch.full((1, pitch), 0xEE, dtype=torch.uint8, device="cuda")[:, :cols]
    assert codes.stride() == (pitch, 1)
    return codes, torch.full((ps.opt_scales_bytes(1, cols),), 0xEE, dtype=torch.uint8, device="cuda")


def same(a, b):
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def in_lines(rows, cols):
    codes, scales = ps.e4m3_storage(rows, cols)
    scales.fill_(0xEE)
    return codes, scales


@pytest.mark.parametrize("cols,pitch", ROWS)
def test_quantize_and_dequantize(cols, pitch):
    x = matrix(1, cols, "f32", 3)
    pair, lines = one_row(cols, pitch), in_lines(1, cols)
    ps.opt_quantize(x, *pair)
    ps.opt_quantize(x, *lines)
    same(pair, lines)
    v = torch.from_numpy(ref.values(*lines)).cuda()
    for dtype in ("bf16", "f32"):
        for turned in (False, True):
            out, t, want = blank(1, cols, dtype, 3), in_lines(cols, 1), in_lines(cols, 1)
            ps.opt_dequantize(*pair, x=out, **(dict(codes_t=t[0], scales_t=t[1]) if turned else {}))
            assert torch.equal(out, v.to(TD[dtype]))
            if turned:
                ps.opt_quantize(v.float(), None, None, *want)
                same(t, want)
    t, want = in_lines(cols, 1), in_lines(cols, 1)
    ps.opt_dequantize(*pair, codes_t=t[0], scales_t=t[1])
    ps.opt_quantize(v.float(), None, None, *want)
    same(t, want)
    # the transposed operand's own single row
    column, row, want = kept_column(x), one_row(cols, pitch), in_lines(1, cols)
    ps.opt_dequantize(*column, codes_t=row[0], scales_t=row[1])
    ps.opt_quantize(torch.from_numpy(ref.values(*column)).float().t().contiguous().cuda(), *want)
    same(row, want)


def kept_column(x):
    pair = in_lines(x.shape[1], 1)
    ps.opt_quantize(x.t().contiguous(), *pair)
    return pair


@pytest.mark.parametrize("cols,pitch", ROWS + [(1032, 1037)])
def test_gated_and_its_gradients(cols, pitch):
    g, u, dy = (matrix(1, cols, "bf16", 5 + i) for i in range(3))
    pairs = {}
    for make in (lambda: one_row(cols, pitch), lambda: in_lines(1, cols)):
        y, gk, uk = make(), make(), make()
        ps.opt_gated(g, u, codes=y[0], scales=y[1], gate_kept=gk, up_kept=uk)
        dg, du = make(), make()
        t = [in_lines(cols, 1) for _ in range(3)]
        ps.opt_gated_backward(dy, gk, uk, dgate_codes=dg, dup_codes=du, dgate_codes_t=t[0], dup_codes_t=t[1], y_codes_t=t[2])
        rows = [make(), make()]
        ps.opt_gated_backward(dy, gk, uk, dgate_codes=rows[0], dup_codes=rows[1])
        same(rows[0], dg)
        same(rows[1], du)
        pairs.setdefault("all", []).append([y, gk, uk, dg, du] + t)
    for a, b in zip(*pairs["all"]):
        same(a, b)


@pytest.mark.parametrize("heads,dim,pitch", [(3, 64, 193), (5, 100, 501), (2, 96, 1030), (1, 300, 300), (7, 1, 7)])
def test_heads_and_their_gradients(heads, dim, pitch):
    cols = heads * dim
    x, dout, w = matrix(1, cols, "bf16", 8), matrix(1, cols, "bf16", 9), torch.ones(dim, device="cuda")
    got = []
    for pair in (one_row(cols, pitch), in_lines(1, cols)):
        y, dx, dw = blank(1, cols, "bf16"), blank(1, cols, "bf16"), torch.empty(dim, device="cuda")
        ps.opt_head_norm(x, w, y, q_kept=pair)
        ps.opt_head_norm_backward(dout, pair, w, dx, dq_weight=dw)
        got.append((pair, y, dx, dw))
    same(got[0][0], got[1][0])
    assert all(torch.equal(a, b) for a, b in zip(got[0][1:], got[1][1:]))


@pytest.mark.parametrize("n", [1, 37, 300])
def test_product(n):
    """A single row by n: the operand and the output of either orientation."""
    k, pitch = 769, 771
    x = matrix(1, k, "f32", 10)
    b = in_lines(n, k)
    ps.opt_quantize(matrix(n, k, "f32", 11), *b)
    outs = []
    for pair in (one_row(k, pitch), in_lines(1, k)):
        ps.opt_quantize(x, *pair)
        out, other = blank(1, n, "f32"), blank(n, 1, "f32")
        ps.opt_matmul(*pair, *b, out)
        ps.opt_matmul(*b, *pair, other)
        outs.append((out, other))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
