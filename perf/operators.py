"""Cases and plain forms of the training-layer operators: dropout from a
counter-based generator, root-mean-square norm with the residual's addition
(forward and backward), conversion to 8-bit floating point with a scale for
each block of 128, and the product of two matrices held in that form.

``run`` computes one operator either in elementary torch operations in 32 bits
(``own`` false) or through the package's entry points (``own`` true);
``exact`` gives the same outputs from the definitions in 64 bits.

Definitions shared by all of them
  dropout   element i of a tensor of n (rows x cols, in row-major order
            whatever the row stride) is kept iff its 16-bit draw is at least
            T = round(65536 p), and a kept value is multiplied by
            65536 / (65536 - T).  Draws come from Philox4x32-10, key = seed,
            counter = (g low 32, g high 32 | 2^31, tensor index, step low 32)
            for g = i / 8; element 8g + j takes word j / 2, its low half for
            even j and its high half for odd j.
  block     1 x 128 elements along the contraction (the last one of a row may
  scales    be shorter), or 128 x 128 for weights.  The scale is 2^e with e
            the smallest integer for which the block's largest magnitude over
            2^e is at most 448, not below -127; it is held as the byte e + 127
            and the values over 2^e as E4M3, rounded to nearest.
  tiles     scale bytes of a rows x cols operand are held in tiles of 128 rows
            by 4 blocks (512 bytes; tiles of a row panel one after another):
            row r, block b at 512 ((r / 128) ceil(B / 4) + b / 4)
            + 16 (r mod 32) + 4 ((r / 32) mod 4) + b mod 4.
"""
import math

import numpy as np
import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_MASK = 0xFFFFFFFF
EPS = 1e-5


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # the residual branch of one new token at width 4096: launch latency
        dict(name="dropout_token", op="dropout", rows=1, cols=4096, dtype="bf16", residual=True, p=0.1, pad=0),
        # the same branch over a training batch of 16,384 tokens, forward (its backward is the
        # call without a residual): the memory-bound end
        dict(name="dropout_batch", op="dropout", rows=16384, cols=4096, dtype="bf16", residual=True, p=0.1, pad=0),
        # one token's norm in front of an 8-bit product, serving
        dict(name="norm_token", op="rms_norm", rows=1, cols=4096, dtype="bf16", weight="f32", out="e4m3",
             residual=True, p=0.0, pad=0),
        # a training batch: branch dropout, residual sum, norm and 8-bit output in one pass
        dict(name="norm_batch", op="rms_norm", rows=16384, cols=4096, dtype="bf16", weight="f32", out="e4m3",
             residual=True, p=0.1, pad=0),
        # fp32 activations of an odd width and an odd number of rows, cut out of wider rows
        dict(name="norm_odd_f32", op="rms_norm", rows=1023, cols=769, dtype="f32", weight="f32", out="both",
             residual=False, p=0.0, pad=3),
        # the backward pass of norm_batch on half its tokens, with the gradient that comes down the
        # residual stream, the branch's gradient and the weight's
        dict(name="norm_grad_batch", op="rms_norm_backward", rows=8192, cols=4096, dtype="bf16", weight="f32",
             dh_in=True, p=0.1, pad=0),
        # the backward pass over a short odd fp32 batch of GPT-2's width and one
        dict(name="norm_grad_odd_f32", op="rms_norm_backward", rows=301, cols=769, dtype="f32", weight="f32",
             dh_in=False, p=0.0, pad=0),
        # a weight of the Llama-3-8B list (the up projection), both orientations, once per step
        dict(name="quantize_weight", op="quantize", rows=14336, cols=4096, dtype="f32", block=128, both=True, pad=0),
        # an incoming gradient of a ragged batch, both orientations (for the two backward products)
        dict(name="quantize_grad", op="quantize", rows=8191, cols=1024, dtype="bf16", block=1, both=True, pad=0),
        # one token through the up projection: the weight's bytes are the time
        dict(name="matmul_token", op="matmul", m=1, n=14336, k=4096, out="bf16", block=128, addend=False),
        # a training batch through the up projection
        dict(name="matmul_batch", op="matmul", m=8192, n=14336, k=4096, out="bf16", block=128, addend=False),
        # a key projection's weight gradient over a ragged batch, added to an fp32 gradient
        dict(name="matmul_weight_grad", op="matmul", m=1024, n=4096, k=8191, out="f32", block=1, addend=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["dropout", "rms_norm", "rms_norm_backward", "quantize", "matmul"])
    if op == "matmul":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 1, 14336), _log(rng, 1, 14336)
            if m * n * k <= 8192 * 14336 * 4096:
                break
        out = rng.choice(["bf16", "f32"])
        return dict(op=op, m=m, n=n, k=k, out=out, block=rng.choice([1, 128]), addend=rng.random() < 0.4)
    limit = {"dropout": 1 << 26, "rms_norm": 1 << 26, "rms_norm_backward": 1 << 25, "quantize": 14336 * 4096}[op]
    while True:
        rows, cols = _log(rng, 1, 16384), _log(rng, 1, 16384)
        if rng.random() < 0.5:
            cols = -(-cols // 128) * 128
        if rows * cols <= limit:
            break
    dtype, pad, p = rng.choice(["bf16", "f32"]), rng.choice([0, 0, 0, 5, 64]), rng.choice([0.0, 0.1, 0.35])
    if op == "dropout":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.5, p=max(p, 0.05), pad=pad)
    if op == "rms_norm":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, weight=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["same", "e4m3", "both"]), residual=rng.random() < 0.6, p=p, pad=pad)
    if op == "rms_norm_backward":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, weight=rng.choice(["bf16", "f32"]),
                    dh_in=rng.random() < 0.6, p=p, pad=pad)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, block=rng.choice([1, 128]), both=rng.random() < 0.6, pad=pad)


# ------------------------------------------------------------------ the inputs
def _normal(gen, rows, cols, dtype, std, pad=0):
    """rows x cols values cut out of rows that are `pad` elements longer."""
    t = torch.empty(rows, cols + pad, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return t.to(_TORCH[dtype])[:, :cols]


def _activations(gen, rows, cols, dtype, pad=0):
    """Unit values with a few channels twenty times the rest, as residual streams have."""
    t = torch.empty(rows, cols + pad, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    t[:, 7 % (cols + pad)::512] *= 20.0
    return t.to(_TORCH[dtype])[:, :cols]


def _codes(rows, cols):
    """Storage of E4M3 codes: rows of a 16-byte pitch."""
    return torch.zeros(rows, -(-max(cols, 1) // 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]


def _scales(rows, cols):
    return torch.zeros(-(-rows // 128) * -(-cols // 512) * 512, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    s = dict(case=case, seed=int(seed) * 0x9E3779B97F4A7C15 % (1 << 64), tensor=3, step=int(seed) % 1000 + 1)
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scales"] = _codes(m, k), _scales(m, k)
        s["b"], s["b_scales"] = _codes(n, k), _scales(n, k)
        for x, std, block, codes, scales in ((_activations(gen, m, k, "f32"), 1.0, 1, s["a"], s["a_scales"]),
                                             (_normal(gen, n, k, "f32", 0.02), 1.0, case["block"], s["b"], s["b_scales"])):
            c, e = _quantize(x, block)
            codes.copy_(c.view(torch.uint8))
            scales.copy_(_tiled(e))
        s["out"] = torch.empty(m, n, dtype=_TORCH[case["out"]], device="cuda")
        s["addend"] = _normal(gen, m, n, case["out"], 1.0) if case["addend"] else None
        return s
    rows, cols, dtype, pad = case["rows"], case["cols"], case["dtype"], case["pad"]
    new = lambda: torch.empty(rows, cols, dtype=_TORCH[dtype], device="cuda")  # noqa: E731
    if op == "dropout":
        s["x"] = _activations(gen, rows, cols, dtype, pad)
        s["residual"] = _activations(gen, rows, cols, dtype) if case["residual"] else None
        s["y"] = new()
    elif op == "rms_norm":
        s["x"] = _activations(gen, rows, cols, dtype, pad)
        s["residual"] = _activations(gen, rows, cols, dtype) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * _normal(gen, 1, cols, "f32", 1.0)[0]).to(_TORCH[case["weight"]])
        s["h"] = new() if case["residual"] or case["p"] > 0 else None
        s["y"] = new() if case["out"] in ("same", "both") else None
        s["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        quant = case["out"] in ("e4m3", "both")
        s["codes"], s["scales"] = (_codes(rows, cols), _scales(rows, cols)) if quant else (None, None)
    elif op == "rms_norm_backward":
        s["h"] = _activations(gen, rows, cols, dtype, pad)
        s["dy"] = _normal(gen, rows, cols, dtype, 1e-2)
        s["weight"] = (1.0 + 0.1 * _normal(gen, 1, cols, "f32", 1.0)[0]).to(_TORCH[case["weight"]])
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dh_in"] = _normal(gen, rows, cols, dtype, 1e-2) if case["dh_in"] else None
        s["dh"], s["dx"] = new(), new() if case["p"] > 0 else None
        s["dweight"] = torch.empty(cols, dtype=torch.float32, device="cuda")
    else:
        s["x"] = _normal(gen, rows, cols, dtype, 0.02 if case["block"] == 128 else 1e-3, pad)
        s["codes"], s["scales"] = _codes(rows, cols), _scales(rows, cols)
        s["codes_t"], s["scales_t"] = (_codes(cols, rows), _scales(cols, rows)) if case["both"] else (None, None)
    return s


# ------------------------------------------------------------- the plain forms
def _keep(n, p, s):
    """The kept elements as booleans, and the factor of the kept ones."""
    g = torch.arange(-(-n // 8), dtype=torch.int64, device="cuda")
    c0, c1, c2, c3 = g & _MASK, (g >> 32) | (1 << 31), torch.full_like(g, s["tensor"]), torch.full_like(g, s["step"] & _MASK)
    k0, k1 = s["seed"] & _MASK, s["seed"] >> 32
    for _ in range(10):      # Philox4x32-10; 64-bit products wrap, their halves are taken from the bits
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & _MASK) ^ c1 ^ k0, p1 & _MASK, ((p0 >> 32) & _MASK) ^ c3 ^ k1, p0 & _MASK
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    w = torch.stack([c0, c1, c2, c3], -1)
    draws = torch.stack([w & 0xFFFF, w >> 16], -1).reshape(-1)[:n]
    t = int(round(65536 * p))
    return draws >= t, 65536.0 / (65536 - t) if t < 65536 else 0.0


def _dropped(x, p, s):
    """Dropout of x (32 bits), by its elements' places in row-major order."""
    if p == 0:
        return x
    keep, factor = _keep(x.numel(), p, s)
    return torch.where(keep.view(x.shape), x * factor, torch.zeros_like(x))


def _tiled(e):
    """Scale bytes [rows, blocks] in tiles of 128 rows by 4 blocks."""
    rows, blocks = e.shape
    pr, pb = -(-rows // 128), -(-blocks // 4)
    full = torch.zeros(pr * 128, pb * 4, dtype=torch.uint8, device=e.device)
    full[:rows, :blocks] = e
    return full.view(pr, 4, 32, pb, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(tiles, rows, blocks):
    pr, pb = -(-rows // 128), -(-blocks // 4)
    return tiles.view(pr, pb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(pr * 128, pb * 4)[:rows, :blocks]


def _quantize(x, block):
    """E4M3 values and scale bytes [rows, blocks] of x (32 bits)."""
    rows, cols = x.shape
    blocks, groups = -(-cols // 128), -(-rows // block)
    full = torch.zeros(groups * block, blocks * 128, dtype=torch.float32, device=x.device)
    full[:rows, :cols] = x
    v = full.view(groups, block, blocks, 128)
    top = v.abs().amax(dim=(1, 3))
    frac, power = torch.frexp(top / 448.0)
    e = torch.where(top > 0, power - (frac <= 0.5).to(power.dtype), torch.full_like(power, -127)).clamp(-127, 127)
    inverse = ((127 - e) << 23).view(torch.float32)                # 2^-e; e is never above 120
    codes = (v * inverse[:, None, :, None]).reshape(groups * block, blocks * 128)[:rows, :cols].to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).repeat_interleave(block, 0)[:rows]


def _values(codes, scales):
    """The values that E4M3 codes and their scales stand for, in 32 bits."""
    rows, cols = codes.shape
    e = _untiled(scales, rows, -(-cols // 128)).to(torch.int32)
    scale = torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, 1)[:, :cols]


def _coded(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "dropout":
        y = _dropped(s["x"].float(), case["p"], s)
        return {"y": (y + s["residual"].float() if s["residual"] is not None else y).to(s["x"].dtype)}
    if op == "rms_norm":
        h = _dropped(s["x"].float(), case["p"], s)
        if s["residual"] is not None:
            h = h + s["residual"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["weight"].float()
        got = {"rstd": rstd}
        if s["h"] is not None:
            got["h"] = h.to(s["x"].dtype)
        if s["y"] is not None:
            got["y"] = y.to(s["x"].dtype)
        if s["codes"] is not None:
            codes, e = _quantize(y, 1)
            got["codes"], got["scales"] = _coded(codes, _tiled(e))
        return got
    if op == "rms_norm_backward":
        dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        g = dy * s["weight"].float()
        dh = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
        if s["dh_in"] is not None:
            dh = dh + s["dh_in"].float()
        got = {"dh": dh.to(s["h"].dtype), "dweight": (dy * h * rstd).sum(0)}
        if case["p"] > 0:
            got["dx"] = _dropped(dh, case["p"], s).to(s["h"].dtype)
        return got
    if op == "quantize":
        x = s["x"].float()
        codes, e = _quantize(x, case["block"])
        got = dict(zip(("codes", "scales"), _coded(codes, _tiled(e))))
        if case["both"]:
            codes, e = _quantize(x.t(), case["block"])
            got["codes_t"], got["scales_t"] = _coded(codes, _tiled(e))
        return got
    out = torch.matmul(_values(s["a"], s["a_scales"]), _values(s["b"], s["b_scales"]).t())
    if s["addend"] is not None:
        out = out + s["addend"].float()
    return {"out": out.to(s["out"].dtype)}


# ------------------------------------------------------- the package's own calls
def _own(s):
    import precision_states_gb300 as ps
    case, op = s["case"], s["case"]["op"]
    if op == "matmul":
        ps.opt_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], addend=s["addend"])
        return {"out": s["out"]}
    if op == "quantize":
        ps.opt_quantize(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"], block_rows=case["block"])
        got = dict(zip(("codes", "scales"), _coded(s["codes"], s["scales"])))
        if case["both"]:
            got["codes_t"], got["scales_t"] = _coded(s["codes_t"], s["scales_t"])
        return got
    draws = dict(p=case["p"], seed=s["seed"], tensor_index=s["tensor"], step=s["step"])
    if op == "dropout":
        ps.opt_dropout(s["x"], s["y"], residual=s["residual"], **draws)
        return {"y": s["y"]}
    if op == "rms_norm":
        ps.opt_rms_norm(s["x"], s["weight"], eps=EPS, y=s["y"], rstd=s["rstd"], residual=s["residual"], h=s["h"],
                        codes=s["codes"], scales=s["scales"], **draws)
        got = {k: s[k] for k in ("rstd", "h", "y") if s[k] is not None}
        if s["codes"] is not None:
            got["codes"], got["scales"] = _coded(s["codes"], s["scales"])
        return got
    ps.opt_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"], dh_in=s["dh_in"], dx=s["dx"],
                             dweight=s["dweight"], **draws)
    return {k: s[k] for k in ("dh", "dweight", "dx") if s[k] is not None}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    held = lambda rows, cols: rows * cols + rows * -(-cols // 128)  # noqa: E731  (codes and scale bytes)
    if op == "matmul":
        m, n, k, out = case["m"], case["n"], case["k"], _SIZE[case["out"]]
        return {"bytes": held(m, k) + held(n, k) + m * n * out * (2 if case["addend"] else 1), "flops": 2 * m * n * k}
    rows, cols, es = case["rows"], case["cols"], _SIZE[case["dtype"]]
    n = rows * cols
    if op == "dropout":
        return {"bytes": n * es * (3 if case["residual"] else 2), "flops": 2 * n}
    if op == "rms_norm":
        moved = n * es * (1 + case["residual"] + (case["residual"] or case["p"] > 0) + (case["out"] != "e4m3"))
        moved += held(rows, cols) if case["out"] != "same" else 0
        return {"bytes": moved + cols * _SIZE[case["weight"]] + 4 * rows, "flops": 6 * n}
    if op == "rms_norm_backward":
        moved = n * es * (3 + case["dh_in"] + (case["p"] > 0))
        return {"bytes": moved + cols * (_SIZE[case["weight"]] + 4) + 4 * rows, "flops": 10 * n}
    return {"bytes": n * es + held(rows, cols) + (held(cols, rows) if case["both"] else 0), "flops": 3 * n}


# -------------------------------------------- the definitions in 64 bits, apart
def _exact_factors(n, p, seed, tensor, step):
    """Each element's factor (0 or 65536 / (65536 - T)) in float64, by numpy."""
    t = int(round(65536 * p))
    out = np.zeros(-(-n // 8) * 8)
    m32 = np.uint64(_MASK)
    for at in range(0, len(out) // 8, 1 << 20):
        g = np.arange(at, min(at + (1 << 20), len(out) // 8), dtype=np.uint64)
        c = [g & m32, (g >> np.uint64(32)) | np.uint64(1 << 31), np.full_like(g, tensor), np.full_like(g, step & _MASK)]
        k = [seed & _MASK, seed >> 32]
        for _ in range(10):
            a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
            c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m32]
            k = [(k[0] + 0x9E3779B9) & _MASK, (k[1] + 0xBB67AE85) & _MASK]
        for j in range(8):
            draws = (c[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
            out[8 * at + j:8 * (at + len(g)):8] = draws >= t
    return out[:n] * (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _exact_quantized(y, block):
    """Values over their scale, not rounded, and the tiled scales, both float64."""
    rows, cols = y.shape
    y2 = torch.nn.functional.pad(y, (0, -cols % 128, 0, -rows % block))
    top = y2.abs().unflatten(0, (-1, block)).unflatten(2, (-1, 128)).amax((1, 3))
    # the smallest e with top <= 448 2^e, found by comparison from the logarithm's floor
    e = torch.floor(torch.log2(top.clamp_min(1e-300) / 448.0)).clamp(-127, 127)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    scale = torch.exp2(e).repeat_interleave(block, 0)[:rows]
    over = y / scale.repeat_interleave(128, 1)[:, :cols]
    r = torch.arange(rows, device=y.device)[:, None]
    b = torch.arange(scale.shape[1], device=y.device)[None, :]
    panel = -(-scale.shape[1] // 4)
    at = 512 * ((r // 128) * panel + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4
    tiles = torch.full((-(-rows // 128) * panel * 512,), 2.0 ** -127, dtype=torch.float64, device=y.device)
    tiles[at.reshape(-1)] = scale.reshape(-1)
    return over, tiles


def _exact_values(codes, scales):
    """E4M3 bytes and tiled scale bytes as float64 values, from the formats' bits."""
    rows, cols = codes.shape
    u = codes.to(torch.int64)
    field, frac = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(field > 0, (1 + frac / 8) * torch.exp2(field.double() - 7), frac * 2.0 ** -9)
    r = torch.arange(rows, device=codes.device)[:, None]
    b = torch.arange(cols, device=codes.device)[None, :] // 128
    at = 512 * ((r // 128) * -(-cols // 512) + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4
    return torch.where(u >= 128, -mag, mag) * torch.exp2(scales[at].double() - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        out = _exact_values(s["a"], s["a_scales"]) @ _exact_values(s["b"], s["b_scales"]).T
        return {"out": out if s["addend"] is None else out + s["addend"].double()}
    if op == "quantize":
        x = s["x"].double()
        got = dict(zip(("codes", "scales"), _exact_quantized(x, case["block"])))
        if case["both"]:
            got["codes_t"], got["scales_t"] = _exact_quantized(x.T.contiguous(), case["block"])
        return got
    p, factors = case["p"], 1.0
    if p > 0:
        f = _exact_factors(case["rows"] * case["cols"], p, s["seed"], s["tensor"], s["step"])
        factors = torch.from_numpy(f).to("cuda").view(case["rows"], case["cols"])
    if op == "rms_norm_backward":
        dy, h, rstd = s["dy"].double(), s["h"].double(), s["rstd"].double()[:, None]
        g = dy * s["weight"].double()
        dh = rstd * g - rstd ** 3 / case["cols"] * h * (g * h).sum(1, keepdim=True)
        if s["dh_in"] is not None:
            dh += s["dh_in"].double()
        got = {"dh": dh, "dweight": (dy * (h * rstd)).sum(0)}
        if p > 0:
            got["dx"] = dh * factors
        return got
    h = s["x"].double() * factors
    if s["residual"] is not None:
        h = h + s["residual"].double()
    if op == "dropout":
        return {"y": h}
    rstd = (h.square().mean(1) + EPS) ** -0.5
    y = h * rstd[:, None] * s["weight"].double()
    got = {"rstd": rstd}
    if s["h"] is not None:
        got["h"] = h
    if s["y"] is not None:
        got["y"] = y
    if s["codes"] is not None:
        got["codes"], got["scales"] = _exact_quantized(y, 1)
    return got
