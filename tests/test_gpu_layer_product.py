"""GPU tests of the block-scaled product's forms: many tiles per pair of CTAs,
each form by name, and the waits of each."""
import pytest
import torch

import precision_states_gb300 as ps

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def integers(rows, k, seed):
    """Small integers and their codes with scales, both exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float()
    codes, scales = ps.e4m3_storage(rows, k)
    ps.opt_quantize(x, codes, scales)
    return x, codes, scales


def check_exact(m, n, k, out, addend, pad, repeats=3):
    """Integers of at most 9 k < 2^24: every partial sum is exact in fp32, so every
    element of the product is, and a BF16 one is the exact sum rounded once."""
    x, a, sa = integers(m, k, 1)
    y, b, sb = integers(n, k, 2)
    want, c = x @ y.T, None
    if addend:
        g = torch.Generator(device="cuda").manual_seed(3)
        c = torch.randint(-200, 201, (m, n + pad), generator=g, device="cuda").to(TD[out])[:, :n]
        want += c
    want = want.to(TD[out])
    d = torch.empty(m, n + pad, dtype=TD[out], device="cuda")
    for _ in range(repeats):
        d.fill_(float("nan"))
        ps.opt_matmul(a, sa, b, sb, d[:, :n], addend=c)
        wrong = (d[:, :n] != want).sum().item()
        assert wrong == 0, f"{wrong} of {m * n} elements"
        assert pad == 0 or torch.isnan(d[:, n:]).all(), "wrote between the rows"
    assert ps.opt_layer_status() == 0


@pytest.mark.parametrize("out,addend,pad", [("bf16", False, 0), ("f32", False, 0), ("bf16", True, 0), ("f32", True, 0),
                                            ("bf16", False, 3), ("f32", True, 3)])
@pytest.mark.parametrize("m,n,k", [(30000, 576, 256), (24576, 640, 256), (65536, 300, 512), (131072, 576, 512),
                                   (65536, 300, 1024), (66000, 320, 128), (800, 14001, 256), (800, 14001, 1000),
                                   (1000, 14336, 128)])
def test_output_warps_at_different_speeds(m, n, k, out, addend, pad):
    """Several tiles per pair whose output warps have unequal work (a ragged last
    column or row of tiles leaves some of them nothing to store): no warp's release
    of a tile counts for another tile's, so no accumulator is overwritten early."""
    check_exact(m, n, k, out, addend, pad)


@pytest.mark.parametrize("k", [(1 << 31) - 1, (1 << 31) - 2047, (1 << 31) - 2048])
def test_few_rows_at_the_greatest_depths(k):
    """Powers of two at the ends of a row of over two thousand million codes, with scale 1."""
    pitch = 1 << 31
    a = torch.zeros(1, pitch, dtype=torch.uint8, device="cuda")
    b = torch.zeros(2, pitch, dtype=torch.uint8, device="cuda")
    scales = torch.full((ps.opt_scales_bytes(1, k),), 127, dtype=torch.uint8, device="cuda")
    one, two, four = 0x38, 0x40, 0x48                          # E4M3
    for at in (0, 2047, 1 << 30, k - 2049, k - 17, k - 1):
        a[0, at] = two
    b[0, 0], b[0, k - 2049], b[0, k - 1] = one, four, one
    b[1, 1 << 30], b[1, k - 17] = two, four
    a[0, k:], b[:, k:] = 0x7F, 0x7F                            # NaN beyond the depth
    out = torch.empty(1, 2, device="cuda")
    ps.opt_matmul(a[:, :k], scales, b[:, :k], scales, out)
    assert out.tolist() == [[12.0, 12.0]]
    ps.opt_matmul(b[:, :k], scales, a[:, :k], scales, out.view(2, 1))
    assert out.tolist() == [[12.0, 12.0]]
