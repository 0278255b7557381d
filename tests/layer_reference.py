"""The training-layer operators' definitions in float64 and numpy, for the
tests: dropout factors from Philox4x32-10, block scales found by comparison,
scale tiles, and the values that codes stand for.  Test infrastructure only."""
import numpy as np
import torch

import oracle


def factors(rows, cols, p, seed, tensor_index, step):
    """Each element's factor (0 or 65536 / (65536 - T)), with the CPU oracle's generator."""
    t = int(np.rint(65536 * p))
    if t == 0:
        return np.ones((rows, cols))
    n = rows * cols
    words = np.array([oracle.philox4x32_10([g & 0xFFFFFFFF, (g >> 32) | 0x80000000, tensor_index, step],
                                           [seed & 0xFFFFFFFF, seed >> 32]) for g in range(-(-n // 8))],
                     dtype=np.int64).reshape(-1)
    draws = np.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:n]
    return np.where(draws >= t, 65536.0 / max(65536 - t, 1), 0.0).reshape(rows, cols)


def block_exponents(x, block_rows):
    """e for each row and 128-element block of x (float64): the smallest e >= -127
    whose 448 2^e holds the block's largest finite magnitude."""
    rows, cols = x.shape
    out = np.empty((rows, -(-cols // 128)), dtype=np.int64)
    mag = np.where(np.isfinite(x), np.abs(x), 0.0)
    for r0 in range(0, rows, block_rows):
        for b in range(out.shape[1]):
            top = mag[r0:r0 + block_rows, 128 * b:128 * b + 128].max()
            e = -127
            if top > 448.0 * 2.0 ** -127:
                e = int(np.floor(np.log2(top / 448.0))) - 1
                while 448.0 * 2.0 ** e < top:
                    e += 1
                e = max(e, -127)
            out[r0:r0 + block_rows, b] = e
    return out


def tile_places(rows, blocks):
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    return 512 * ((r // 128) * -(-blocks // 4) + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4


def scale_bytes_of(scales, rows, cols):
    """Scale bytes [rows, blocks] out of the tiles."""
    return scales.cpu().numpy()[tile_places(rows, -(-cols // 128))].astype(np.int64)


def values(codes, scales):
    """float64 values of codes with tiled scales (CPU numpy)."""
    rows, cols = codes.shape
    c = codes.cpu().contiguous().view(torch.float8_e4m3fn).to(torch.float64).numpy()
    e = scale_bytes_of(scales, rows, cols) - 127
    return c * 2.0 ** np.repeat(e, 128, 1)[:, :cols].astype(np.float64)


def encode(x, e):
    """E4M3 bytes of float32 x over its blocks' 2^e; infinities and NaN as NaN."""
    rows, cols = x.shape
    # exact scaling: in float64, then to float32 (a value that rounds there is far below E4M3's grid)
    v = x.astype(np.float64) * 2.0 ** -np.repeat(e, 128, 1)[:, :cols].astype(np.float64)
    v = np.where(np.isfinite(x), v, np.nan)
    got = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    got[~np.isfinite(x)] = 0x7F
    return got
