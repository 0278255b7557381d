"""GPU tests of the block-scaled product's forms: many tiles per pair of CTAs,
each form by name, and the waits of each."""
import pytest
import torch

import precision_states_gb300 as ps

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def integers(rows, k, seed, lines=True):
    """Small integers times a power of two up to 8 that differs by row and block, and
    their codes with scales, both exact.  lines: rows of codes start on 128 bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float()
    place = torch.arange(rows, device="cuda")[:, None] + 3 * (torch.arange(k, device="cuda") // 128)[None, :]
    x *= torch.exp2((place % 4).float())
    codes, scales = ps.e4m3_storage(rows, k)
    scales.fill_(0xFF)                                        # NaN wherever the quantizer does not write
    if not lines:
        pitch = -(-k // 16) * 16
        codes = torch.full((rows, pitch + (16 if pitch % 128 == 0 else 0)), 0x7F, dtype=torch.uint8, device="cuda")[:, :k]
    ps.opt_quantize(x, codes, scales)
    return x, codes, scales


def check_exact(m, n, k, out, addend, pad, repeats=3, lines=True, form=None):
    """Every partial sum is an integer of at most 576 k < 2^24, exact in fp32, so every
    element of the product is exact, and a BF16 one is the exact sum rounded once."""
    assert 576 * k < 1 << 24
    x, a, sa = integers(m, k, 1, lines)
    y, b, sb = integers(n, k, 2, lines)
    if form is not None:
        got = ps.opt_matmul_form(a, b)
        assert got[:4] + (min(got[4], 3),) == form, f"another form now: {got}"
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


# (CTAs of a tile, its columns, parts of the depth, rows of b, tiles in turn: 3 for more), a shape
# that takes it on a GB300, and whether its rows of codes start on lines
FORMS = [
    ((1, 16, 1, 0, 1), (12, 14, 100), True), ((1, 16, 1, 1, 3), (16, 50000, 300), True), ((1, 16, 1, 0, 3), (50000, 12, 300), True),
    ((1, 16, 2, 1, 1), (12, 5353, 4000), True), ((1, 16, 2, 0, 1), (5353, 12, 4000), True), ((1, 16, 4, 1, 1), (9, 18, 1809), False),
    ((1, 16, 8, 0, 1), (12, 16, 5000), True),
    ((1, 32, 1, 1, 1), (17, 33, 18), True), ((1, 32, 1, 1, 3), (30, 50000, 300), True), ((1, 32, 1, 0, 3), (50000, 30, 300), True), ((1, 32, 2, 1, 1), (20, 5300, 4000), True),
    ((1, 32, 2, 0, 1), (5300, 20, 4000), True), ((1, 32, 4, 1, 1), (30, 40, 2100), False), ((1, 32, 8, 1, 1), (30, 40, 5000), True),
    ((1, 64, 1, 1, 1), (35, 70, 16), True), ((1, 64, 1, 1, 3), (60, 50000, 300), True), ((1, 64, 1, 0, 3), (50000, 60, 300), True), ((1, 64, 2, 0, 1), (5245, 40, 5000), True),
    ((1, 64, 4, 1, 1), (60, 4600, 4000), True), ((1, 64, 8, 1, 1), (60, 100, 5000), True),
    ((1, 128, 1, 0, 1), (100, 70, 300), True), ((1, 128, 1, 0, 2), (3096, 1329, 40), True), ((1, 128, 1, 0, 3), (824, 5560, 904), True),
    ((1, 128, 2, 0, 1), (66, 4711, 5055), False), ((1, 128, 4, 0, 1), (300, 700, 8000), True), ((1, 128, 8, 0, 1), (256, 256, 4000), True),
    # more clusters than the device holds at once
    ((1, 16, 2, 1, 1), (9, 19550, 18991), False), ((1, 64, 2, 0, 1), (19842, 33, 16254), False),
    ((2, 128, 1, 0, 1), (100, 4711, 6000), True), ((2, 128, 1, 0, 2), (3989, 1142, 784), False), ((2, 128, 1, 0, 3), (4000, 1700, 1300), True),
    ((2, 256, 1, 0, 1), (1000, 4096, 5000), True), ((2, 256, 1, 0, 2), (2048, 4096, 400), True), ((2, 256, 1, 0, 3), (2602, 3410, 260), False)]


@pytest.mark.parametrize("out,addend,pad", [("bf16", False, 0), ("f32", True, 0), ("bf16", True, 3), ("f32", False, 3)])
@pytest.mark.parametrize("form,size,lines", FORMS)
def test_forms(form, size, lines, out, addend, pad):
    check_exact(*size, out, addend, pad, repeats=1, lines=lines, form=form)


def test_every_form_is_tested():
    """Each tile with one and with several in turn, each split."""
    have = {f[:3] + (f[4] > 1,) for f, _, _ in FORMS}
    assert have == {(1, n, s, False) for n in (16, 32, 64, 128) for s in (1, 2, 4, 8)} | {
        (1, n, 1, True) for n in (16, 32, 64, 128)} | {(2, n, 1, many) for n in (128, 256) for many in (False, True)}


@pytest.mark.parametrize("form,size,lines", [f for f in FORMS if f[0][4] != 2 and f[1][0] * f[1][1] < 10_000_000])
def test_wait_drill_of_each_form(form, size, lines):
    """A product whose waits run out reports it once, writes nothing and leaves the
    next one as it is: single CTAs, clusters that leave together, and pairs."""
    m, n, k = size
    x, a, sa = integers(m, k, 4, lines)
    y, b, sb = integers(n, k, 5, lines)
    assert ps.opt_matmul_form(a, b)[:3] == form[:3]
    out = torch.full((m, n), 7.0, device="cuda")
    assert ps.opt_layer_status() == 0
    ps.opt_matmul(a, sa, b, sb, out, wait_drill=True)
    assert ps.opt_layer_status() == ps.OPT_FLAG_WAIT_TIMEOUT and (out == 7).all()
    assert ps.opt_layer_status() == 0
    ps.opt_matmul(a, sa, b, sb, out)
    assert torch.equal(out, x @ y.T) and ps.opt_layer_status() == 0


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
