"""Cases and plain forms of the operators between a block's products, and of the
activations that a training step keeps in 8 bits: the gated activation and its
gradients, the norm of each query and key head with the position rotation and
its gradients, and what becomes of kept codes in the backward pass.

``run`` computes one operator either in elementary torch operations in 32 bits
(``own`` false) or through the package's entry points (``own`` true);
``exact`` gives the same outputs from the definitions in 64 bits.

Definitions
  kept      a rows x cols matrix as E4M3 codes with a scale for each 1 x 128 of
            a row (the row's last block may be shorter): 2^e with e the smallest
            integer, not below -127, for which the block's largest magnitude over
            2^e is at most 448, held as the byte e + 127; codes are the values
            over 2^e rounded to nearest.
  tiles     scale bytes of a rows x cols operand are held in tiles of 128 rows
            by 4 blocks (512 bytes; tiles of a row panel one after another):
            row r, block b at 512 ((r / 128) ceil(B / 4) + b / 4)
            + 16 (r mod 32) + 4 ((r / 32) mod 4) + b mod 4.
  turned    the transposed operand of a matrix: cols x rows codes, with blocks of
            128 along the matrix's rows.
  gated     y = f(gate) up; f(g) = g s(g) with s the logistic function of g
            (silu) or of 2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu_tanh), the
            normal distribution's (gelu), or [g > 0] (relu).
  heads     per row and head of `dim` elements: n = x w / sqrt(mean(x^2) + eps);
            the first `rot` elements of n are rotated in pairs, (i, i + rot / 2)
            or (2 i, 2 i + 1), by the angle whose cosine and sine stand at the
            row's position in two tables.
"""
import math

import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token between a block's up and down projections (Llama-3-8B's width): launch latency
        dict(name="gated_token", op="gated", rows=1, cols=14336, dtype="bf16", act="silu", up=True, out="codes",
             kept=False, pad=0),
        # a training batch: the down projection's operand, and both inputs kept in 8 bits
        dict(name="gated_batch", op="gated", rows=8192, cols=14336, dtype="bf16", act="silu", up=True, out="codes",
             kept=True, pad=0),
        # fp32 activations of an odd width cut out of wider rows, GELU, plain output
        dict(name="gated_odd_f32", op="gated", rows=1023, cols=2303, dtype="f32", act="gelu", up=True, out="plain",
             kept=False, pad=3),
        # the backward pass of gated_batch: every operand of the six products behind and before it, from what was kept
        dict(name="gated_grad_batch", op="gated_backward", rows=8192, cols=14336, dtype="bf16", act="silu", up=True,
             source="kept", out="turned", pad=0),
        # the gradients of a short batch of an odd width, plain in and out
        dict(name="gated_grad_odd", op="gated_backward", rows=515, cols=2303, dtype="bf16", act="gelu_tanh", up=True,
             source="plain", out="plain", pad=0),
        # a projection's kept input (16,384 tokens of width 4096) as its weight gradient's operand
        dict(name="turn_batch", op="dequantize", rows=16384, cols=4096, dtype="bf16", plain=False, turned=True, pad=0),
        # a ragged batch of GPT-2's width and one: plain values again, and the turned operand
        dict(name="dequantize_odd", op="dequantize", rows=8191, cols=769, dtype="bf16", plain=True, turned=True, pad=0),
        # one new token's query and key heads (Llama-3-8B: 32 and 8 of 128): launch latency
        dict(name="heads_token", op="head_norm", rows=1, q_heads=32, k_heads=8, dim=128, rot=128, interleaved=False,
             dtype="bf16", weight="f32", kept=False, packed=True),
        # a training batch of 16,384 tokens, the projections' outputs kept in 8 bits
        dict(name="heads_batch", op="head_norm", rows=16384, q_heads=32, k_heads=8, dim=128, rot=128, interleaved=False,
             dtype="bf16", weight="f32", kept=True, packed=False),
        # GPT-2's 12 heads of 64 inside rows of 2304, fp32, half of each head rotated in neighbouring pairs
        dict(name="heads_odd_f32", op="head_norm", rows=1023, q_heads=12, k_heads=12, dim=64, rot=32, interleaved=True,
             dtype="f32", weight="f32", kept=False, packed=True),
        # the backward pass of heads_batch on half its tokens, from what was kept
        dict(name="heads_grad_batch", op="head_norm_backward", rows=8192, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, dtype="bf16", weight="f32", source="kept", packed=False),
        # the gradients of a short batch with heads of 96, plain
        dict(name="heads_grad_odd", op="head_norm_backward", rows=301, q_heads=8, k_heads=2, dim=96, rot=96,
             interleaved=False, dtype="bf16", weight="bf16", source="plain", packed=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gated", "gated_backward", "dequantize", "head_norm", "head_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gated", "gated_backward", "dequantize"):
        limit = {"gated": 1 << 26, "gated_backward": 1 << 25, "dequantize": 1 << 26}[op]
        while True:
            rows, cols = _log(rng, 1, 16384), _log(rng, 1, 16384)
            if rng.random() < 0.5:
                cols = -(-cols // 128) * 128
            if rows * cols <= limit:
                break
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype, pad=rng.choice([0, 0, 0, 5, 64]))
        if op == "dequantize":
            plain, turned = rng.choice([(True, False), (False, True), (True, True)])
            return dict(case, plain=plain, turned=turned)
        case.update(act=rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]), up=rng.random() < 0.8)
        if op == "gated":
            return dict(case, out=rng.choice(["plain", "codes", "both"]), kept=rng.random() < 0.5)
        return dict(case, source=rng.choice(["kept", "plain"]), out=rng.choice(["plain", "codes", "turned"]))
    dim = rng.choice([32, 48, 64, 64, 80, 96, 128, 128, 128, 160, 192, 256, 100, 33])
    rot = rng.choice([dim, dim, dim // 2, dim // 4, 0]) // 2 * 2
    q_heads = _log(rng, 1, 64)
    k_heads = rng.choice([0, 1, q_heads, max(q_heads // 4, 1)])
    limit = (1 << 25) if op == "head_norm" else (1 << 24)
    rows = _log(rng, 1, max(min(16384, limit // ((q_heads + k_heads) * dim)), 2))
    case = dict(op=op, rows=rows, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, interleaved=rng.random() < 0.4,
                dtype=dtype, weight=rng.choice(["bf16", "f32"]), packed=rng.random() < 0.5)
    if op == "head_norm":
        return dict(case, kept=rng.random() < 0.5)
    return dict(case, source=rng.choice(["kept", "plain"]))


# ------------------------------------------------------------------ the inputs
def _normal(gen, rows, cols, dtype, std, pad=0):
    """rows x cols values cut out of rows that are `pad` elements longer."""
    t = torch.empty(rows, cols + pad, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return t.to(_TORCH[dtype])[:, :cols]


def _uneven(gen, rows, cols, dtype, pad=0):
    """Unit values with a few channels ten times the rest, as a projection's outputs have."""
    t = torch.empty(rows, cols + pad, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    t[:, 5 % (cols + pad)::384] *= 10.0
    return t.to(_TORCH[dtype])[:, :cols]


def _storage(rows, cols):
    """Storage of a kept matrix: codes in rows of a 16-byte pitch, and their scale tiles."""
    codes = torch.zeros(rows, -(-max(cols, 1) // 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]
    return codes, torch.zeros(-(-rows // 128) * -(-cols // 512) * 512, dtype=torch.uint8, device="cuda")


def _keep(x):
    """x kept in 8 bits, as an earlier call left it."""
    codes, scales = _storage(*x.shape)
    c, s = _coded(x.float())
    codes.copy_(c.view(torch.uint8))
    scales.copy_(s.view(torch.uint8))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)
    s = dict(case=case)
    op, rows, dtype = case["op"], case["rows"], case["dtype"]
    if op in ("head_norm", "head_norm_backward"):
        dim, heads, rot = case["dim"], (case["q_heads"], case["k_heads"]), case["rot"]
        table = 8192
        angle = torch.arange(table, dtype=torch.float64, device="cuda")[:, None] * torch.exp(
            torch.arange(rot // 2, dtype=torch.float64, device="cuda") * (-2.0 * math.log(5e5) / max(rot, 1)))
        s["cos"], s["sin"] = (torch.cos(angle).float(), torch.sin(angle).float()) if rot else (None, None)
        # sequences packed behind one another, each from a position of its own
        start = int(torch.randint(0, table // 2, (1,), generator=gen, device="cuda").item())
        s["positions"] = (torch.arange(rows, device="cuda") + start) % table if rot else None
        widths = [h * dim for h in heads]
        if case["packed"]:      # both inside a projection's rows, with as many value heads as key heads
            x = _uneven(gen, rows, sum(widths) + widths[1], dtype)
            xs = [x[:, :widths[0]], x[:, widths[0]:sum(widths)]]
        else:
            xs = [_uneven(gen, rows, w, dtype) if w else None for w in widths]
        for name, x, h in zip(("q", "k"), xs, heads):
            if h == 0:
                s[name] = None
                continue
            s[name] = x
            s[name + "_weight"] = (1.0 + 0.1 * _normal(gen, 1, dim, "f32", 1.0)[0]).to(_TORCH[case["weight"]])
            if op == "head_norm":
                s[name + "_out"] = torch.empty(rows, h * dim, dtype=_TORCH[dtype], device="cuda")
                s[name + "_kept"] = _storage(rows, h * dim) if case["kept"] else None
            else:
                if case["source"] == "kept":
                    s[name] = _keep(x)
                s["d" + name + "_out"] = _normal(gen, rows, h * dim, dtype, 1e-2)
                s["d" + name] = torch.empty(rows, h * dim, dtype=_TORCH[dtype], device="cuda")
                s["d" + name + "_weight"] = torch.empty(dim, dtype=torch.float32, device="cuda")
        return s
    cols, pad = case["cols"], case["pad"]
    new = lambda: torch.empty(rows, cols, dtype=_TORCH[dtype], device="cuda")  # noqa: E731
    if op == "dequantize":
        s["codes"], s["scales"] = _keep(_uneven(gen, rows, cols, "f32"))
        s["x"] = torch.empty(rows, cols + pad, dtype=_TORCH[dtype], device="cuda")[:, :cols] if case["plain"] else None
        s["turned"] = _storage(cols, rows) if case["turned"] else (None, None)
        return s
    gate = _uneven(gen, rows, cols, dtype, pad)
    up = _uneven(gen, rows, cols, dtype, pad) if case["up"] else None
    if op == "gated":
        s["gate"], s["up"] = gate, up
        s["y"] = new() if case["out"] in ("plain", "both") else None
        s["coded"] = _storage(rows, cols) if case["out"] in ("codes", "both") else (None, None)
        s["gate_kept"] = _storage(rows, cols) if case["kept"] else None
        s["up_kept"] = _storage(rows, cols) if case["kept"] and case["up"] else None
        return s
    keep = _keep if case["source"] == "kept" else lambda x: x
    s["gate"], s["up"] = keep(gate), keep(up) if case["up"] else None
    s["dy"] = _normal(gen, rows, cols, dtype, 1e-2)
    for name in ("dgate", "dup") if case["up"] else ("dgate",):
        s[name] = new() if case["out"] == "plain" else None
        s[name + "_codes"] = _storage(rows, cols) if case["out"] != "plain" else None
        s[name + "_codes_t"] = _storage(cols, rows) if case["out"] == "turned" else None
    s["y_codes_t"] = _storage(cols, rows) if case["out"] == "turned" else None
    return s


# ------------------------------------------------------------- the plain forms
def _coded(x):
    """x (32 bits) as E4M3 values and tiled scales, in the types that torch has for them."""
    rows, cols = x.shape
    blocks = -(-cols // 128)
    full = torch.zeros(rows, blocks * 128, dtype=torch.float32, device=x.device)
    full[:, :cols] = x
    v = full.view(rows, blocks, 128)
    top = v.abs().amax(dim=2)
    frac, power = torch.frexp(top / 448.0)
    e = torch.where(top > 0, power - (frac <= 0.5).to(power.dtype), torch.full_like(power, -127)).clamp(-127, 127)
    inverse = ((127 - e) << 23).view(torch.float32)                # 2^-e; e is never above 120
    codes = (v * inverse[:, :, None]).view(rows, blocks * 128)[:, :cols].to(torch.float8_e4m3fn)
    pr, pb = -(-rows // 128), -(-blocks // 4)
    tiles = torch.zeros(pr * 128, pb * 4, dtype=torch.uint8, device=x.device)
    tiles[:rows, :blocks] = (e + 127).to(torch.uint8)
    tiles = tiles.view(pr, 4, 32, pb, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return codes, tiles.view(torch.float8_e8m0fnu)


def _values(codes, tiles):
    """The values that codes and their scales stand for, in 32 bits."""
    rows, cols = codes.shape
    pr, pb = -(-rows // 128), -(-cols // 512)
    e = tiles.view(pr, pb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(pr * 128, pb * 4)[:rows].to(torch.int32)
    scale = torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, 1)[:, :cols]


def _plain_of(x):
    """A matrix or a kept one, in 32 bits."""
    return _values(*x) if isinstance(x, tuple) else x.float()


def _put(got, name, x):
    got[name], got[name + "_scales"] = _coded(x)


def _activation(g, act):
    """f(g) and its derivative, in g's type."""
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "gelu":
        s = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * s, s + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5
    if act == "silu":
        z, dz = g, 1.0
    else:
        c = 2.0 * (2.0 / math.pi) ** 0.5
        z, dz = c * (g + 0.044715 * g * g * g), c * (1.0 + 3 * 0.044715 * g * g)
    s, not_s = 1.0 / (1.0 + torch.exp(-z)), 1.0 / (1.0 + torch.exp(z))
    return g * s, s + g * s * not_s * dz


def _rotated(n, s, back):
    """Heads [rows, heads, dim] turned by their rows' angles, or back."""
    rot = s["case"]["rot"]
    if rot == 0:
        return n
    c, sn = (t[s["positions"]][:, None, :] for t in (s["cos"], s["sin"]))
    if back:
        sn = -sn
    first, second, rest = n[..., :rot // 2], n[..., rot // 2:rot], n[..., rot:]
    if s["case"]["interleaved"]:
        first, second = n[..., 0:rot:2], n[..., 1:rot:2]
    a, b = first * c - second * sn, second * c + first * sn
    turned = torch.stack([a, b], -1).flatten(-2) if s["case"]["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _plain_heads(s, name):
    case = s["case"]
    rows, dim, dtype = case["rows"], case["dim"], _TORCH[case["dtype"]]
    x = _plain_of(s[name]).reshape(rows, -1, dim)
    w = s[name + "_weight"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(2, keepdim=True) + EPS)
    if case["op"] == "head_norm":
        got = {name: _rotated(x * rstd * w, s, False).reshape(rows, -1).to(dtype)}
        if case["kept"]:
            _put(got, name + "_kept", x.reshape(rows, -1))
        return got
    g = _rotated(s["d" + name + "_out"].float().reshape(rows, -1, dim), s, True)
    t = g * w
    dx = rstd * (t - x * (rstd * rstd * (t * x).mean(2, keepdim=True)))
    return {"d" + name: dx.reshape(rows, -1).to(dtype), "d" + name + "_weight": (g * x * rstd).sum((0, 1))}


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op in ("head_norm", "head_norm_backward"):
        got = _plain_heads(s, "q")
        if s["k"] is not None:
            got.update(_plain_heads(s, "k"))
        return got
    got = {}
    if op == "dequantize":
        v = _values(s["codes"], s["scales"])
        if case["plain"]:
            got["x"] = v.to(s["x"].dtype)
        if case["turned"]:
            _put(got, "turned", v.t())
        return got
    dtype = _TORCH[case["dtype"]]
    gate, up = _plain_of(s["gate"]), _plain_of(s["up"]) if case["up"] else None
    f, df = _activation(gate, case["act"])
    y = f * up if case["up"] else f
    if op == "gated":
        if s["y"] is not None:
            got["y"] = y.to(dtype)
        if s["coded"][0] is not None:
            _put(got, "codes", y)
        if case["kept"]:
            _put(got, "gate_kept", gate)
        if case["kept"] and case["up"]:
            _put(got, "up_kept", up)
        return got
    dy = s["dy"].float()
    dgate = dy * df * up if case["up"] else dy * df
    _put_gradient(got, "dgate", dgate, case)
    if case["up"]:
        _put_gradient(got, "dup", dy * f, case)
    if case["out"] == "turned":
        _put(got, "y_codes_t", y.t())
    return got


def _put_gradient(got, name, x, case):
    if case["out"] == "plain":
        got[name] = x.to(_TORCH[case["dtype"]])
    else:
        _put(got, name + "_codes", x)
    if case["out"] == "turned":
        _put(got, name + "_codes_t", x.t())


# ------------------------------------------------------- the package's own calls
def _show(got, name, pair):
    """A kept output in the types that torch has for its codes and scales."""
    if pair is not None and pair[0] is not None:
        got[name], got[name + "_scales"] = pair[0].view(torch.float8_e4m3fn), pair[1].view(torch.float8_e8m0fnu)


def _own(s):
    import precision_states_gb300 as ps
    case, op, got = s["case"], s["case"]["op"], {}
    if op in ("head_norm", "head_norm_backward"):
        both = s["k"] is not None
        how = dict(eps=EPS, cos=s["cos"], sin=s["sin"], positions=s["positions"], interleaved=case["interleaved"])
        if op == "head_norm":
            more = dict(k=s["k"], k_weight=s["k_weight"], k_out=s["k_out"], k_kept=s["k_kept"]) if both else {}
            ps.opt_head_norm(s["q"], s["q_weight"], s["q_out"], q_kept=s["q_kept"], **more, **how)
            got["q"] = s["q_out"]
            _show(got, "q_kept", s["q_kept"])
            if both:
                got["k"] = s["k_out"]
                _show(got, "k_kept", s["k_kept"])
            return got
        more = dict(dk_out=s["dk_out"], k=s["k"], k_weight=s["k_weight"], dk=s["dk"],
                    dk_weight=s["dk_weight"]) if both else {}
        ps.opt_head_norm_backward(s["dq_out"], s["q"], s["q_weight"], s["dq"], dq_weight=s["dq_weight"], **more, **how)
        got["dq"], got["dq_weight"] = s["dq"], s["dq_weight"]
        if both:
            got["dk"], got["dk_weight"] = s["dk"], s["dk_weight"]
        return got
    if op == "dequantize":
        ps.opt_dequantize(s["codes"], s["scales"], x=s["x"], codes_t=s["turned"][0], scales_t=s["turned"][1])
        if s["x"] is not None:
            got["x"] = s["x"]
        _show(got, "turned", s["turned"])
        return got
    if op == "gated":
        ps.opt_gated(s["gate"], s["up"], activation=case["act"], y=s["y"], codes=s["coded"][0], scales=s["coded"][1],
                     gate_kept=s["gate_kept"], up_kept=s["up_kept"])
        if s["y"] is not None:
            got["y"] = s["y"]
        _show(got, "codes", s["coded"])
        _show(got, "gate_kept", s["gate_kept"])
        _show(got, "up_kept", s["up_kept"])
        return got
    more = dict(dup=s["dup"], dup_codes=s["dup_codes"], dup_codes_t=s["dup_codes_t"]) if case["up"] else {}
    ps.opt_gated_backward(s["dy"], s["gate"], s["up"], activation=case["act"], dgate=s["dgate"],
                          dgate_codes=s["dgate_codes"], dgate_codes_t=s["dgate_codes_t"], y_codes_t=s["y_codes_t"], **more)
    if s["dgate"] is not None:
        got["dgate"] = s["dgate"]
    _show(got, "dgate_codes", s["dgate_codes"])
    _show(got, "dgate_codes_t", s["dgate_codes_t"])
    if case["up"]:
        if s["dup"] is not None:
            got["dup"] = s["dup"]
        _show(got, "dup_codes", s["dup_codes"])
        _show(got, "dup_codes_t", s["dup_codes_t"])
    _show(got, "y_codes_t", s["y_codes_t"])
    return got


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, rows, es = case["op"], case["rows"], _SIZE[case["dtype"]]
    held = lambda r, c: r * c + r * -(-c // 128)  # noqa: E731  (codes and scale bytes)
    if op in ("head_norm", "head_norm_backward"):
        moved = flops = 0
        for heads in (case["q_heads"], case["k_heads"]):
            cols = heads * case["dim"]
            if op == "head_norm":
                moved += rows * cols * 2 * es + (held(rows, cols) if case["kept"] else 0)
            else:
                moved += rows * cols * 2 * es + (held(rows, cols) if case["source"] == "kept" else rows * cols * es)
                moved += case["dim"] * 4 * (heads > 0)
            moved += case["dim"] * _SIZE[case["weight"]] * (heads > 0)
            flops += rows * cols * (8 if op == "head_norm" else 16)
        # each row's position, and the tables' lines of its angles (each line once)
        return {"bytes": moved + (8 * rows + 4 * case["rot"] * min(rows, 8192) if case["rot"] else 0), "flops": flops}
    cols = case["cols"]
    n = rows * cols
    if op == "dequantize":
        return {"bytes": held(rows, cols) + (n * es if case["plain"] else 0) + (held(cols, rows) if case["turned"] else 0),
                "flops": 3 * n}
    inputs = 2 if case["up"] else 1
    if op == "gated":
        moved = n * es * inputs + (n * es if case["out"] != "codes" else 0) + (held(rows, cols) if case["out"] != "plain" else 0)
        return {"bytes": moved + (inputs * held(rows, cols) if case["kept"] else 0), "flops": 8 * n}
    moved = n * es + inputs * (held(rows, cols) if case["source"] == "kept" else n * es)
    moved += inputs * (n * es if case["out"] == "plain" else held(rows, cols))
    return {"bytes": moved + ((inputs + 1) * held(cols, rows) if case["out"] == "turned" else 0), "flops": 20 * n}


# -------------------------------------------- the definitions in 64 bits, apart
def _places(rows, blocks, device):
    """The tiles' place of each row's and block's scale byte."""
    r, b = torch.arange(rows, device=device)[:, None], torch.arange(blocks, device=device)[None, :]
    return 512 * ((r // 128) * -(-blocks // 4) + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4


def _exact_coded(got, name, y):
    """Values over their scale, not rounded, and the tiled scales, both float64."""
    rows, cols = y.shape
    top = torch.nn.functional.pad(y, (0, -cols % 128)).abs().unflatten(1, (-1, 128)).amax(2)
    # the smallest e with top <= 448 2^e, found by comparison from the logarithm's floor
    e = torch.floor(torch.log2(top.clamp_min(1e-300) / 448.0)).clamp(-127, 127)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    scale = torch.exp2(e)
    got[name] = y / scale.repeat_interleave(128, 1)[:, :cols]
    tiles = torch.full((-(-rows // 128) * -(-cols // 512) * 512,), 2.0 ** -127, dtype=torch.float64, device=y.device)
    tiles[_places(rows, scale.shape[1], y.device).reshape(-1)] = scale.reshape(-1)
    got[name + "_scales"] = tiles


def _exact_of(x):
    """A matrix or a kept one as float64, the latter from the formats' bits."""
    if not isinstance(x, tuple):
        return x.double()
    codes, tiles = x
    u = codes.to(torch.int64)
    field, frac = (u >> 3) & 15, (u & 7).double()
    mag = torch.where(field > 0, (1 + frac / 8) * torch.exp2(field.double() - 7), frac * 2.0 ** -9)
    rows, cols = codes.shape
    e = tiles[_places(rows, -(-cols // 128), codes.device)].double() - 127
    return torch.where(u >= 128, -mag, mag) * torch.exp2(e).repeat_interleave(128, 1)[:, :cols]


def _exact_share(g, act):
    """s(g) with f(g) = g s(g), and f'(g)."""
    if act == "relu":
        return (g > 0).double(), (g > 0).double()
    if act == "gelu":
        share = torch.special.ndtr(g)
        return share, share + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        share = torch.sigmoid(g)
        return share, share * (1 + g * torch.sigmoid(-g))
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    th = torch.tanh(inner)
    slope = math.sqrt(2 / math.pi) * (1 + 0.134145 * g.square())
    return torch.sigmoid(2 * inner), torch.sigmoid(2 * inner) + 0.5 * g * (1 - th.square()) * slope


def _exact_heads(s, got, name):
    """By complex numbers: each pair as one, each row's angle as a factor."""
    case = s["case"]
    rows, dim, rot = case["rows"], case["dim"], case["rot"]
    x = _exact_of(s[name]).reshape(rows, -1, dim)
    w = s[name + "_weight"].double()
    rstd = (x.square().mean(2, keepdim=True) + EPS) ** -0.5
    if rot:
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"]][:, None, :]

    def turned(n, by):
        if not rot:
            return n
        out = n.clone()
        if case["interleaved"]:
            z = torch.complex(n[..., 0:rot:2], n[..., 1:rot:2]) * by
            out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * by
            out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
        return out

    if case["op"] == "head_norm":
        got[name] = turned(x * rstd * w, turn if rot else None).reshape(rows, -1)
        if case["kept"]:
            _exact_coded(got, name + "_kept", x.reshape(rows, -1))
        return
    g = turned(s["d" + name + "_out"].double().reshape(rows, -1, dim), turn.conj() if rot else None)
    dx = rstd * g * w - rstd ** 3 / dim * x * (g * w * x).sum(2, keepdim=True)
    got["d" + name] = dx.reshape(rows, -1)
    got["d" + name + "_weight"] = (g * (x * rstd)).sum((0, 1))


def exact(case, seed):
    s = prepare(case, seed)
    op, got = case["op"], {}
    if op in ("head_norm", "head_norm_backward"):
        _exact_heads(s, got, "q")
        if s["k"] is not None:
            _exact_heads(s, got, "k")
        return got
    if op == "dequantize":
        v = _exact_of((s["codes"], s["scales"]))
        if case["plain"]:
            got["x"] = v
        if case["turned"]:
            _exact_coded(got, "turned", v.T.contiguous())
        return got
    gate, up = _exact_of(s["gate"]), _exact_of(s["up"]) if case["up"] else 1.0
    share, slope = _exact_share(gate, case["act"])
    if op == "gated":
        y = gate * share * up
        if s["y"] is not None:
            got["y"] = y
        if s["coded"][0] is not None:
            _exact_coded(got, "codes", y)
        if case["kept"]:
            _exact_coded(got, "gate_kept", gate)
            if case["up"]:
                _exact_coded(got, "up_kept", up)
        return got
    dy = s["dy"].double()
    outs = [("dgate", dy * slope * up)] + ([("dup", dy * gate * share)] if case["up"] else [])
    for name, x in outs:
        if case["out"] == "plain":
            got[name] = x
        else:
            _exact_coded(got, name + "_codes", x)
        if case["out"] == "turned":
            _exact_coded(got, name + "_codes_t", x.T.contiguous())
    if case["out"] == "turned":
        _exact_coded(got, "y_codes_t", (gate * share * up).T.contiguous())
    return got
