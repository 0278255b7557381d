"""Python binding of the training-layer operators (include/opt_layer.h):
dropout, residual RMS norm and its gradients, conversion to E4M3 with a scale
for each block of 128 and back, the product of two matrices held in that form,
the gated activation and the heads' norm with rotation, and their gradients from
inputs that are kept in it.

Argument marshalling and shape checks only; the functions carry the C names
and write into tensors that the caller owns.  A matrix argument is a CUDA
tensor on the current device whose last dimension is contiguous: a 2-d tensor
of any row stride, or a contiguous tensor of any other shape, taken as rows of
its last dimension.  A kept matrix, or another operand in 8 bits that an argument
names as one, is a pair (codes, scales) as e4m3_storage gives it.  Wrong shapes
and dtypes, and numbers that their C types do not hold, raise ValueError;
everything else is checked by the library (OptError).
"""
from __future__ import annotations

import ctypes
import struct

_c = ctypes
_vp, _i64, _u64, _i32, _u32, _f32, _f64 = (_c.c_void_p, _c.c_int64, _c.c_uint64, _c.c_int32, _c.c_uint32,
                                           _c.c_float, _c.c_double)


class opt_dropout_args(_c.Structure):
    _fields_ = [("d_x", _vp), ("d_residual", _vp), ("d_y", _vp),
                ("x_pitch", _i64), ("residual_pitch", _i64), ("y_pitch", _i64),
                ("rows", _i64), ("cols", _i64), ("p", _f64), ("seed", _u64), ("step", _i64),
                ("tensor_index", _u32), ("dtype", _i32)]


class opt_rms_norm_args(_c.Structure):
    _fields_ = [("d_x", _vp), ("d_residual", _vp), ("d_weight", _vp), ("d_h", _vp), ("d_y", _vp), ("d_rstd", _vp),
                ("d_codes", _vp), ("d_scales", _vp),
                ("x_pitch", _i64), ("residual_pitch", _i64), ("h_pitch", _i64), ("y_pitch", _i64),
                ("codes_pitch", _i64), ("rows", _i64), ("cols", _i64), ("p", _f64), ("seed", _u64), ("step", _i64),
                ("tensor_index", _u32), ("dtype", _i32), ("weight_dtype", _i32), ("eps", _f32)]


class opt_rms_norm_backward_args(_c.Structure):
    _fields_ = [("d_dy", _vp), ("d_h", _vp), ("d_weight", _vp), ("d_rstd", _vp), ("d_dh_in", _vp), ("d_dh", _vp),
                ("d_dx", _vp), ("d_dweight", _vp), ("d_workspace", _vp),
                ("dy_pitch", _i64), ("h_pitch", _i64), ("dh_in_pitch", _i64), ("dh_pitch", _i64), ("dx_pitch", _i64),
                ("workspace_bytes", _i64), ("rows", _i64), ("cols", _i64), ("p", _f64), ("seed", _u64),
                ("step", _i64), ("tensor_index", _u32), ("dtype", _i32), ("weight_dtype", _i32), ("reserved", _i32)]


class opt_quantize_args(_c.Structure):
    _fields_ = [("d_x", _vp), ("d_codes", _vp), ("d_scales", _vp), ("d_codes_t", _vp), ("d_scales_t", _vp),
                ("x_pitch", _i64), ("codes_pitch", _i64), ("codes_t_pitch", _i64), ("rows", _i64), ("cols", _i64),
                ("dtype", _i32), ("block_rows", _i32)]


class opt_dequantize_args(_c.Structure):
    _fields_ = [("d_codes", _vp), ("d_scales", _vp), ("d_x", _vp), ("d_codes_t", _vp), ("d_scales_t", _vp),
                ("codes_pitch", _i64), ("x_pitch", _i64), ("codes_t_pitch", _i64), ("rows", _i64), ("cols", _i64),
                ("dtype", _i32), ("reserved", _i32)]


class opt_gated_args(_c.Structure):
    _fields_ = [("d_gate", _vp), ("d_up", _vp), ("d_y", _vp), ("d_codes", _vp), ("d_scales", _vp), ("d_gate_codes", _vp),
                ("d_gate_scales", _vp), ("d_up_codes", _vp), ("d_up_scales", _vp),
                ("gate_pitch", _i64), ("up_pitch", _i64), ("y_pitch", _i64), ("codes_pitch", _i64),
                ("gate_codes_pitch", _i64), ("up_codes_pitch", _i64), ("rows", _i64), ("cols", _i64),
                ("dtype", _i32), ("activation", _i32)]


class opt_gated_backward_args(_c.Structure):
    _fields_ = [("d_dy", _vp), ("d_gate", _vp), ("d_gate_scales", _vp), ("d_up", _vp), ("d_up_scales", _vp),
                ("d_dgate", _vp), ("d_dup", _vp), ("d_dgate_codes", _vp), ("d_dgate_scales", _vp),
                ("d_dgate_codes_t", _vp), ("d_dgate_scales_t", _vp), ("d_dup_codes", _vp), ("d_dup_scales", _vp),
                ("d_dup_codes_t", _vp), ("d_dup_scales_t", _vp), ("d_y_codes_t", _vp), ("d_y_scales_t", _vp),
                ("dy_pitch", _i64), ("gate_pitch", _i64), ("up_pitch", _i64), ("dgate_pitch", _i64), ("dup_pitch", _i64),
                ("dgate_codes_pitch", _i64), ("dgate_codes_t_pitch", _i64), ("dup_codes_pitch", _i64),
                ("dup_codes_t_pitch", _i64), ("y_codes_t_pitch", _i64), ("rows", _i64), ("cols", _i64),
                ("dtype", _i32), ("activation", _i32)]


class opt_head_norm_args(_c.Structure):
    _fields_ = [("d_q", _vp), ("d_q_weight", _vp), ("d_q_out", _vp), ("d_q_codes", _vp), ("d_q_scales", _vp),
                ("d_k", _vp), ("d_k_weight", _vp), ("d_k_out", _vp), ("d_k_codes", _vp), ("d_k_scales", _vp),
                ("d_cos", _vp), ("d_sin", _vp), ("d_positions", _vp),
                ("q_pitch", _i64), ("q_out_pitch", _i64), ("q_codes_pitch", _i64), ("k_pitch", _i64), ("k_out_pitch", _i64),
                ("k_codes_pitch", _i64), ("rows", _i64), ("q_heads", _i64), ("k_heads", _i64), ("dim", _i64), ("rot", _i64),
                ("positions", _i64), ("dtype", _i32), ("weight_dtype", _i32), ("flags", _i32), ("eps", _f32)]


class opt_head_norm_backward_args(_c.Structure):
    _fields_ = [("d_dq_out", _vp), ("d_q", _vp), ("d_q_scales", _vp), ("d_q_weight", _vp), ("d_dq", _vp), ("d_dq_weight", _vp),
                ("d_dk_out", _vp), ("d_k", _vp), ("d_k_scales", _vp), ("d_k_weight", _vp), ("d_dk", _vp), ("d_dk_weight", _vp),
                ("d_cos", _vp), ("d_sin", _vp), ("d_positions", _vp), ("d_workspace", _vp),
                ("dq_out_pitch", _i64), ("q_pitch", _i64), ("dq_pitch", _i64), ("dk_out_pitch", _i64), ("k_pitch", _i64),
                ("dk_pitch", _i64), ("workspace_bytes", _i64), ("rows", _i64), ("q_heads", _i64), ("k_heads", _i64),
                ("dim", _i64), ("rot", _i64), ("positions", _i64), ("dtype", _i32), ("weight_dtype", _i32), ("flags", _i32),
                ("eps", _f32)]


class opt_matmul_args(_c.Structure):
    _fields_ = [("d_a", _vp), ("d_a_scales", _vp), ("d_b", _vp), ("d_b_scales", _vp), ("d_addend", _vp),
                ("d_out", _vp), ("a_pitch", _i64), ("b_pitch", _i64), ("addend_pitch", _i64), ("out_pitch", _i64),
                ("m", _i64), ("n", _i64), ("k", _i64), ("out_dtype", _i32), ("flags", _i32)]


# the C ABI: name -> (restype, argtypes); the argument structs go as packed bytes
SIGS = {
    "opt_scales_bytes": (_i64, [_i64, _i64]),
    "opt_dropout": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_rms_norm": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_rms_norm_backward": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_rms_norm_backward_workspace": (_i64, [_i64, _i64]),
    "opt_quantize": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_dequantize": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_gated": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_gated_backward": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_head_norm": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_head_norm_backward": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_head_norm_backward_workspace": (_i64, [_i64, _i64, _i64, _i64]),
    "opt_matmul": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_matmul_form": (_c.c_int, [_c.c_char_p, _c.POINTER(_i32)]),
    "opt_layer_status": (_c.c_int, [_c.POINTER(_i32), _vp]),
}

OPT_MATMUL_WAIT_DRILL = 1
OPT_HEADS_INTERLEAVED = 1
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1, "gelu": 2, "relu": 3}      # OPT_ACT_*

_CODE = {_vp: "Q", _i64: "q", _u64: "Q", _i32: "i", _u32: "I", _f32: "f", _f64: "d"}


def packer(struct_type):
    """struct.pack for a ctypes argument struct: one call instead of one
    attribute store per field.  Every struct orders its fields so that it has no
    padding."""
    return struct.Struct("=" + "".join(_CODE[t] for _, t in struct_type._fields_)).pack


_pack_dropout = packer(opt_dropout_args)
_pack_rms_norm = packer(opt_rms_norm_args)
_pack_rms_norm_backward = packer(opt_rms_norm_backward_args)
_pack_quantize = packer(opt_quantize_args)
_pack_dequantize = packer(opt_dequantize_args)
_pack_gated = packer(opt_gated_args)
_pack_gated_backward = packer(opt_gated_backward_args)
_pack_head_norm = packer(opt_head_norm_args)
_pack_head_norm_backward = packer(opt_head_norm_backward_args)
_pack_matmul = packer(opt_matmul_args)
_NOT_HELD = (struct.error, OverflowError)      # a number outside its field's type

from . import OPT_BF16, OPT_EUNSUPPORTED, OPT_F32, OptError, _check, _stream_ptr, lib  # noqa: E402


class _Ready:
    """What every call needs, resolved at the first one: the library's functions,
    torch's dtypes and its current device and stream (by their raw forms: a call
    of a small operator takes the GPU two microseconds)."""

    def __init__(self):
        import torch
        L = lib()
        self.dtypes = {torch.float32: OPT_F32, torch.bfloat16: OPT_BF16}
        self.bytes8 = (torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu)
        self.f32, self.int64 = torch.float32, torch.int64
        self.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        self.dropout, self.rms_norm, self.rms_norm_backward = L.opt_dropout, L.opt_rms_norm, L.opt_rms_norm_backward
        self.quantize, self.matmul = L.opt_quantize, L.opt_matmul
        self.dequantize, self.gated, self.gated_backward = L.opt_dequantize, L.opt_gated, L.opt_gated_backward
        self.head_norm, self.head_norm_backward = L.opt_head_norm, L.opt_head_norm_backward


_ready = None


def _get_ready():
    global _ready
    if _ready is None:
        _ready = _Ready()
    return _ready


def _refuse_dtype(t, what):
    raise OptError(OPT_EUNSUPPORTED, f"{what}: dtype {t.dtype}")


def _device(t, what, ready):
    """The tensor's device index, which must be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != ready.device():
        raise ValueError(f"{what} must be a CUDA tensor on the current device")
    return dev


def _matrix(t, what):
    """(rows, cols, pitch) of a matrix argument."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        pitch, step = t.stride()
        if step != 1 and cols > 1 and rows > 0:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        return rows, cols, pitch
    if not t.is_contiguous() or len(shape) == 0:
        raise ValueError(f"{what} must be 2-d with a contiguous last dimension, or contiguous")
    cols = shape[-1]
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return rows, cols, cols


def _like(t, what, rows, cols, dtype, device):
    """(pointer, pitch) of a matrix of the given shape and dtype."""
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{what}: expected {dtype} on cuda:{device}")
    r, c, pitch = _matrix(t, what)
    if r != rows or c != cols:
        raise ValueError(f"{what}: expected {rows} x {cols}, got {tuple(t.shape)}")
    return t.data_ptr(), pitch


def _vector(t, what, n, device, dtype):
    """The pointer of n contiguous elements."""
    if t.dtype != dtype or t.numel() != n or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous elements of {dtype} on cuda:{device}")
    return t.data_ptr()


def _held(codes, scales, what, rows, cols, device, ready):
    """(codes pointer, scales pointer, pitch) of an 8-bit operand."""
    if codes is None or scales is None:
        raise ValueError(f"{what}: codes and scales go together")
    if codes.dtype not in ready.bytes8 or scales.dtype not in ready.bytes8 or codes.get_device() != device:
        raise ValueError(f"{what}: expected 8-bit codes and scales on cuda:{device}")
    r, c, pitch = _matrix(codes, what)
    if r != rows or c != cols:
        raise ValueError(f"{what}: expected codes of {rows} x {cols}, got {tuple(codes.shape)}")
    return codes.data_ptr(), _vector(scales, what, -(-rows // 128) * -(-cols // 512) * 512, device, scales.dtype), pitch


def _pair(kept, what, rows, cols, device, ready):
    """(codes pointer, scales pointer, pitch) of a pair, or zeros without one."""
    if kept is None:
        return 0, 0, 0
    if not isinstance(kept, (tuple, list)) or len(kept) != 2:
        raise ValueError(f"{what}: expected a pair (codes, scales)")
    return _held(kept[0], kept[1], what, rows, cols, device, ready)


def scales_bytes(rows: int, cols: int) -> int:
    """Bytes of the scale tiles of a rows x cols operand (opt_scales_bytes)."""
    return -(-rows // 128) * -(-cols // 512) * 512


def e4m3_storage(rows: int, cols: int, device="cuda"):
    """Zeroed storage of an 8-bit operand: (codes, scales), uint8.  The codes are
    a rows x cols view of rows that are padded to 128 bytes: the calls ask for 16,
    but a product's loads of rows that do not start on lines take up to twice as
    long (773 x 10368 x 8847: 106 us with rows of 8,848 bytes, 61 with 8,960)."""
    import torch
    codes = torch.zeros(rows, -(-max(cols, 1) // 128) * 128, dtype=torch.uint8, device=device)[:, :cols]
    return codes, torch.zeros(scales_bytes(rows, cols), dtype=torch.uint8, device=device)


def opt_scales_bytes(rows: int, cols: int) -> int:
    return _check(lib().opt_scales_bytes(rows, cols), "opt_scales_bytes")


def opt_dropout(x, y, p: float, seed=0, tensor_index=0, step=0, residual=None, stream=None):
    """y = residual + dropout(x); y may be x or residual.  The backward pass is
    the same call on the gradient (same p, seed, tensor_index and step)."""
    ready = _ready or _get_ready()
    dtype = x.dtype
    dt = ready.dtypes.get(dtype)
    if dt is None:
        _refuse_dtype(x, "x")
    dev = _device(x, "x", ready)
    rows, cols, xp = _matrix(x, "x")
    yq, yp = _like(y, "y", rows, cols, dtype, dev)
    rq, rp = (0, 0) if residual is None else _like(residual, "residual", rows, cols, dtype, dev)
    try:
        args = _pack_dropout(x.data_ptr(), rq, yq, xp, rp, yp, rows, cols, p, seed, step, tensor_index, dt)
    except _NOT_HELD as e:
        raise ValueError(f"opt_dropout: {e}") from None
    st = ready.dropout(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_dropout")


def opt_rms_norm(x, weight, eps=1e-5, y=None, rstd=None, residual=None, h=None, codes=None, scales=None, p=0.0,
                 seed=0, tensor_index=0, step=0, stream=None):
    """h = residual + dropout(x), rstd = 1 / sqrt(mean(h^2) + eps) and
    y = h rstd weight, into whichever of h, rstd, y and codes with scales (y as
    E4M3, a scale for each 1 x 128) are given."""
    ready = _ready or _get_ready()
    dtype, wtype = x.dtype, weight.dtype
    dt, wt = ready.dtypes.get(dtype), ready.dtypes.get(wtype)
    if dt is None or wt is None:
        _refuse_dtype(x if dt is None else weight, "x" if dt is None else "weight")
    dev = _device(x, "x", ready)
    rows, cols, xp = _matrix(x, "x")
    wq = _vector(weight, "weight", cols, dev, wtype)
    rq, rp = (0, 0) if residual is None else _like(residual, "residual", rows, cols, dtype, dev)
    hq, hp = (0, 0) if h is None else _like(h, "h", rows, cols, dtype, dev)
    yq, yp = (0, 0) if y is None else _like(y, "y", rows, cols, dtype, dev)
    sq = 0 if rstd is None else _vector(rstd, "rstd", rows, dev, ready.f32)
    cq, eq, cp = ((0, 0, 0) if codes is None and scales is None
                  else _held(codes, scales, "codes", rows, cols, dev, ready))
    try:
        args = _pack_rms_norm(x.data_ptr(), rq, wq, hq, yq, sq, cq, eq, xp, rp, hp, yp, cp, rows, cols, p, seed, step,
                              tensor_index, dt, wt, eps)
    except _NOT_HELD as e:
        raise ValueError(f"opt_rms_norm: {e}") from None
    st = ready.rms_norm(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_rms_norm")


def opt_rms_norm_backward(dy, h, weight, rstd, dh, dh_in=None, dx=None, dweight=None, p=0.0, seed=0, tensor_index=0,
                          step=0, workspace=None, stream=None):
    """Gradients of opt_rms_norm from dy and the stored h and rstd: dh (the
    residual's, with dh_in added), dx = dropout(dh) (the branch's) and dweight
    (fp32).  workspace: a uint8 tensor of opt_rms_norm_backward_workspace(rows,
    cols) bytes for dweight; without one the call takes it from torch's
    allocator."""
    ready = _ready or _get_ready()
    dtype, wtype = h.dtype, weight.dtype
    dt, wt = ready.dtypes.get(dtype), ready.dtypes.get(wtype)
    if dt is None or wt is None:
        _refuse_dtype(h if dt is None else weight, "h" if dt is None else "weight")
    dev = _device(h, "h", ready)
    rows, cols, hp = _matrix(h, "h")
    wq = _vector(weight, "weight", cols, dev, wtype)
    gq, gp = _like(dy, "dy", rows, cols, dtype, dev)
    iq, ip = (0, 0) if dh_in is None else _like(dh_in, "dh_in", rows, cols, dtype, dev)
    oq, op = _like(dh, "dh", rows, cols, dtype, dev)
    xq, xp = (0, 0) if dx is None else _like(dx, "dx", rows, cols, dtype, dev)
    sq = _vector(rstd, "rstd", rows, dev, ready.f32)
    dq = nq = need = 0
    if dweight is not None:
        dq = _vector(dweight, "dweight", cols, dev, ready.f32)
        if workspace is not None:
            need = _given_workspace(workspace, dev)
        elif rows > 512 or rows * cols > 1 << 21:                   # opt_rms_norm_backward_workspace
            need = min(rows, 1024) * (-(-cols // 4) * 4) * 4
            workspace = _workspace(need, dev, stream)
        if need:
            nq = workspace.data_ptr()
    try:
        args = _pack_rms_norm_backward(gq, h.data_ptr(), wq, sq, iq, oq, xq, dq, nq, gp, hp, ip, op, xp, need, rows, cols,
                                       p, seed, step, tensor_index, dt, wt, 0)
    except _NOT_HELD as e:
        raise ValueError(f"opt_rms_norm_backward: {e}") from None
    st = ready.rms_norm_backward(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_rms_norm_backward")


def _given_workspace(t, device):
    """Bytes of a caller's workspace."""
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace: expected contiguous bytes on cuda:{device}")
    return t.numel() * t.element_size()


def _workspace(nbytes, device, stream):
    """Scratch from torch's allocator, out of the pool of the stream that uses it: a
    block of another stream's may still be read or written by work pending there."""
    import torch
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        pointer = _stream_ptr(stream)
        stream = torch.cuda.ExternalStream(0 if pointer == 1 else pointer, device=device)     # 1: the default stream by CUDA's other name
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def opt_rms_norm_backward_workspace(rows: int, cols: int) -> int:
    return _check(lib().opt_rms_norm_backward_workspace(rows, cols), "opt_rms_norm_backward_workspace")


def opt_quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, block_rows=1, stream=None):
    """x to E4M3 codes with a scale for each block of block_rows (1 or 128) x 128:
    as it is (codes, scales) and/or transposed (codes_t of cols x rows,
    scales_t)."""
    ready = _ready or _get_ready()
    dt = ready.dtypes.get(x.dtype)
    if dt is None:
        _refuse_dtype(x, "x")
    dev = _device(x, "x", ready)
    rows, cols, xp = _matrix(x, "x")
    cq, sq, cp = ((0, 0, 0) if codes is None and scales is None
                  else _held(codes, scales, "codes", rows, cols, dev, ready))
    tq, uq, tp = ((0, 0, 0) if codes_t is None and scales_t is None
                  else _held(codes_t, scales_t, "codes_t", cols, rows, dev, ready))
    try:
        args = _pack_quantize(x.data_ptr(), cq, sq, tq, uq, xp, cp, tp, rows, cols, dt, block_rows)
    except _NOT_HELD as e:
        raise ValueError(f"opt_quantize: {e}") from None
    st = ready.quantize(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_quantize")


def opt_dequantize(codes, scales, x=None, codes_t=None, scales_t=None, stream=None):
    """Kept codes as their values (x, float32 or bfloat16) and/or as the transposed
    operand (codes_t of cols x rows, scales_t) with blocks of 128 along the rows."""
    ready = _ready or _get_ready()
    dev = _device(codes, "codes", ready)
    rows, cols, _ = _matrix(codes, "codes")
    cq, sq, cp = _held(codes, scales, "codes", rows, cols, dev, ready)
    dt = OPT_F32
    xq = xp = 0
    if x is not None:
        dt = ready.dtypes.get(x.dtype)
        if dt is None:
            _refuse_dtype(x, "x")
        xq, xp = _like(x, "x", rows, cols, x.dtype, dev)
    tq, uq, tp = ((0, 0, 0) if codes_t is None and scales_t is None
                  else _held(codes_t, scales_t, "codes_t", cols, rows, dev, ready))
    args = _pack_dequantize(cq, sq, xq, tq, uq, cp, xp, tp, rows, cols, dt, 0)
    st = ready.dequantize(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_dequantize")


def _activation(name):
    kind = ACTIVATIONS.get(name)
    if kind is None:
        raise ValueError(f"activation: expected one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return kind


def opt_gated(gate, up=None, activation="silu", y=None, codes=None, scales=None, gate_kept=None, up_kept=None, stream=None):
    """y = f(gate) up (without up: f(gate)) into y and/or codes with scales (E4M3, a
    scale for each 1 x 128), and the inputs into the pairs gate_kept and up_kept for
    the backward pass.  activation: silu, gelu_tanh, gelu or relu."""
    ready = _ready or _get_ready()
    dtype = gate.dtype
    dt = ready.dtypes.get(dtype)
    if dt is None:
        _refuse_dtype(gate, "gate")
    kind = _activation(activation)
    dev = _device(gate, "gate", ready)
    rows, cols, gp = _matrix(gate, "gate")
    uq, up_ = (0, 0) if up is None else _like(up, "up", rows, cols, dtype, dev)
    yq, yp = (0, 0) if y is None else _like(y, "y", rows, cols, dtype, dev)
    cq, sq, cp = ((0, 0, 0) if codes is None and scales is None
                  else _held(codes, scales, "codes", rows, cols, dev, ready))
    gcq, gsq, gcp = _pair(gate_kept, "gate_kept", rows, cols, dev, ready)
    ucq, usq, ucp = _pair(up_kept, "up_kept", rows, cols, dev, ready)
    args = _pack_gated(gate.data_ptr(), uq, yq, cq, sq, gcq, gsq, ucq, usq, gp, up_, yp, cp, gcp, ucp, rows, cols, dt, kind)
    st = ready.gated(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_gated")


def opt_gated_backward(dy, gate, up=None, activation="silu", dgate=None, dup=None, dgate_codes=None, dgate_codes_t=None,
                       dup_codes=None, dup_codes_t=None, y_codes_t=None, stream=None):
    """Gradients of opt_gated from dy, and gate and up as matrices or as the pairs that
    it kept: dgate and dup as matrices, as pairs (dgate_codes, dup_codes), and as
    transposed pairs (dgate_codes_t, dup_codes_t); y again as a transposed pair
    (y_codes_t).  Whichever are given."""
    ready = _ready or _get_ready()
    dtype = dy.dtype
    dt = ready.dtypes.get(dtype)
    if dt is None:
        _refuse_dtype(dy, "dy")
    kind = _activation(activation)
    dev = _device(dy, "dy", ready)
    rows, cols, dp = _matrix(dy, "dy")
    kept = isinstance(gate, (tuple, list))
    if up is not None and isinstance(up, (tuple, list)) != kept:
        raise ValueError("gate and up: both matrices or both kept")
    gsq = usq = 0
    if kept:
        gq, gsq, gp = _pair(gate, "gate", rows, cols, dev, ready)
        uq, usq, up_ = _pair(up, "up", rows, cols, dev, ready)
    else:
        gq, gp = _like(gate, "gate", rows, cols, dtype, dev)
        uq, up_ = (0, 0) if up is None else _like(up, "up", rows, cols, dtype, dev)
    aq, ap = (0, 0) if dgate is None else _like(dgate, "dgate", rows, cols, dtype, dev)
    bq, bp = (0, 0) if dup is None else _like(dup, "dup", rows, cols, dtype, dev)
    acq, asq, acp = _pair(dgate_codes, "dgate_codes", rows, cols, dev, ready)
    atq, auq, atp = _pair(dgate_codes_t, "dgate_codes_t", cols, rows, dev, ready)
    bcq, bsq, bcp = _pair(dup_codes, "dup_codes", rows, cols, dev, ready)
    btq, buq, btp = _pair(dup_codes_t, "dup_codes_t", cols, rows, dev, ready)
    ytq, yuq, ytp = _pair(y_codes_t, "y_codes_t", cols, rows, dev, ready)
    args = _pack_gated_backward(dy.data_ptr(), gq, gsq, uq, usq, aq, bq, acq, asq, atq, auq, bcq, bsq, btq, buq, ytq, yuq,
                                dp, gp, up_, ap, bp, acp, atp, bcp, btp, ytp, rows, cols, dt, kind)
    st = ready.gated_backward(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_gated_backward")


def _heads(t, what, dim):
    """(rows, heads, pitch) of heads of dim elements: a matrix of rows x (heads dim), a
    rows x heads x dim tensor with contiguous heads, or any contiguous one that ends in
    heads x dim."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols, pitch = _matrix(t, what)
        if cols % dim:
            raise ValueError(f"{what}: {cols} columns are not whole heads of {dim}")
        return rows, cols // dim, pitch
    if len(shape) < 3 or shape[-1] != dim:
        raise ValueError(f"{what}: expected rows x heads x {dim}, got {tuple(shape)}")
    if len(shape) == 3 and (dim == 1 or t.stride(2) == 1) and (shape[1] == 1 or t.stride(1) == dim):
        return shape[0], shape[1], t.stride(0)
    if not t.is_contiguous():
        raise ValueError(f"{what}: heads and their elements must be contiguous")
    rows = 1
    for n in shape[:-2]:
        rows *= n
    return rows, shape[-2], shape[-2] * dim


def _like_heads(t, what, rows, heads, dim, dtype, device):
    """(pointer, pitch) of heads of the given number and dtype."""
    if t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{what}: expected {dtype} on cuda:{device}")
    shape = t.shape
    if len(shape) == 2 and shape[0] == rows and shape[1] == heads * dim:
        pitch, step = t.stride()
        if step == 1:                                      # the common case
            return t.data_ptr(), pitch
    r, h, pitch = _heads(t, what, dim)
    if r != rows or h != heads:
        raise ValueError(f"{what}: expected {rows} rows of {heads} heads of {dim}, got {tuple(shape)}")
    return t.data_ptr(), pitch


def _turn(cos, sin, positions, rows, device, ready):
    """(cos, sin and positions pointers, rotated elements, positions in the tables)."""
    if cos is None or sin is None:
        if cos is not None or sin is not None:
            raise ValueError("cos and sin go together")
        if positions is not None:
            raise ValueError("positions: without cos and sin")
        return 0, 0, 0, 0, 0
    shape = cos.shape
    if len(shape) != 2 or sin.shape != shape:
        raise ValueError(f"cos and sin: expected positions x pairs each, got {tuple(shape)} and {tuple(sin.shape)}")
    table, pairs = shape
    f32 = ready.f32
    if (cos.dtype != f32 or sin.dtype != f32 or cos.get_device() != device or sin.get_device() != device
            or not cos.is_contiguous() or not sin.is_contiguous()):
        raise ValueError(f"cos and sin: expected contiguous {f32} on cuda:{device}")
    pq = 0 if positions is None else _vector(positions, "positions", rows, device, ready.int64)
    return cos.data_ptr(), sin.data_ptr(), pq, 2 * pairs, table


def opt_head_norm(q, q_weight, q_out, k=None, k_weight=None, k_out=None, eps=1e-5, cos=None, sin=None, positions=None,
                  interleaved=False, q_kept=None, k_kept=None, stream=None):
    """Each head of q (and of k) over its root mean square, times the weight (whose
    length is a head's), its first elements turned in pairs by the row's angles, into
    q_out and k_out.  cos and sin: float32 tables of positions x pairs; positions: int64,
    a row's place in them (without: its number).  Pairs are an element of the rotated
    part's first half and its second half's, or neighbours (interleaved).  q_kept and
    k_kept: pairs that keep q and k for the backward pass."""
    ready = _ready or _get_ready()
    dtype, wtype = q.dtype, q_weight.dtype
    dt, wt = ready.dtypes.get(dtype), ready.dtypes.get(wtype)
    if dt is None or wt is None:
        _refuse_dtype(q if dt is None else q_weight, "q" if dt is None else "q_weight")
    dev = _device(q, "q", ready)
    dim = q_weight.numel()
    if dim == 0:
        raise ValueError("q_weight: a head has at least one element")
    rows, hq, qp = _heads(q, "q", dim)
    wq = _vector(q_weight, "q_weight", dim, dev, wtype)
    oq, op = _like_heads(q_out, "q_out", rows, hq, dim, dtype, dev)
    cq, sq, cp = _pair(q_kept, "q_kept", rows, hq * dim, dev, ready)
    kq = kp = kwq = koq = kop = kcq = ksq = kcp = hk = 0
    if k is None:
        if not (k_weight is None and k_out is None and k_kept is None):
            raise ValueError("k_weight, k_out and k_kept: without k")
    else:
        if k_weight is None or k_out is None:
            raise ValueError("k: needs k_weight and k_out")
        rk, hk, kp = _heads(k, "k", dim)
        if rk != rows or k.dtype != dtype or k.get_device() != dev:
            raise ValueError(f"k: expected {rows} rows of {dtype} on cuda:{dev}")
        kq = k.data_ptr()
        kwq = _vector(k_weight, "k_weight", dim, dev, wtype)
        koq, kop = _like_heads(k_out, "k_out", rows, hk, dim, dtype, dev)
        kcq, ksq, kcp = _pair(k_kept, "k_kept", rows, hk * dim, dev, ready)
    tc, ts, tp, rot, table = _turn(cos, sin, positions, rows, dev, ready)
    try:
        args = _pack_head_norm(q.data_ptr(), wq, oq, cq, sq, kq, kwq, koq, kcq, ksq, tc, ts, tp, qp, op, cp, kp, kop, kcp, rows,
                               hq, hk, dim, rot, table, dt, wt, OPT_HEADS_INTERLEAVED if interleaved else 0, eps)
    except _NOT_HELD as e:
        raise ValueError(f"opt_head_norm: {e}") from None
    st = ready.head_norm(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_head_norm")


def opt_head_norm_backward(dq_out, q, q_weight, dq, dk_out=None, k=None, k_weight=None, dk=None, dq_weight=None,
                           dk_weight=None, eps=1e-5, cos=None, sin=None, positions=None, interleaved=False, workspace=None,
                           stream=None):
    """Gradients of opt_head_norm from those of its outputs (dq_out, dk_out) and its
    inputs, as matrices or as the pairs that it kept: dq and dk, and the weights'
    (float32).  workspace: a uint8 tensor of opt_head_norm_backward_workspace(...) bytes
    for the weights' gradients; without one the call takes it from torch's allocator."""
    ready = _ready or _get_ready()
    dtype, wtype = dq_out.dtype, q_weight.dtype
    dt, wt = ready.dtypes.get(dtype), ready.dtypes.get(wtype)
    if dt is None or wt is None:
        _refuse_dtype(dq_out if dt is None else q_weight, "dq_out" if dt is None else "q_weight")
    dev = _device(dq_out, "dq_out", ready)
    dim = q_weight.numel()
    if dim == 0:
        raise ValueError("q_weight: a head has at least one element")
    rows, hq, gp = _heads(dq_out, "dq_out", dim)
    kept = isinstance(q, (tuple, list))
    if k is not None and isinstance(k, (tuple, list)) != kept:
        raise ValueError("q and k: both matrices or both kept")

    def given(x, what, heads):
        if kept:
            return _pair(x, what, rows, heads * dim, dev, ready)
        p, pitch = _like_heads(x, what, rows, heads, dim, dtype, dev)
        return p, 0, pitch

    xq, xsq, xp = given(q, "q", hq)
    wq = _vector(q_weight, "q_weight", dim, dev, wtype)
    oq, op = _like_heads(dq, "dq", rows, hq, dim, dtype, dev)
    dwq = 0 if dq_weight is None else _vector(dq_weight, "dq_weight", dim, dev, ready.f32)
    kgq = kgp = kq = ksq = kp = kwq = koq = kop = kdwq = hk = 0
    if dk_out is None:
        if not (k is None and k_weight is None and dk is None and dk_weight is None):
            raise ValueError("k, k_weight, dk and dk_weight: without dk_out")
    else:
        if k is None or k_weight is None or dk is None:
            raise ValueError("dk_out: needs k, k_weight and dk")
        rk, hk, kgp = _heads(dk_out, "dk_out", dim)
        if rk != rows or dk_out.dtype != dtype or dk_out.get_device() != dev:
            raise ValueError(f"dk_out: expected {rows} rows of {dtype} on cuda:{dev}")
        kgq = dk_out.data_ptr()
        kq, ksq, kp = given(k, "k", hk)
        kwq = _vector(k_weight, "k_weight", dim, dev, wtype)
        koq, kop = _like_heads(dk, "dk", rows, hk, dim, dtype, dev)
        kdwq = 0 if dk_weight is None else _vector(dk_weight, "dk_weight", dim, dev, ready.f32)
    tc, ts, tp, rot, table = _turn(cos, sin, positions, rows, dev, ready)
    nq = need = 0
    if dwq or kdwq:
        if workspace is not None:
            need = _given_workspace(workspace, dev)
        else:
            need = min(rows * (hq + hk), 1024) * 8 * dim               # opt_head_norm_backward_workspace
            workspace = _workspace(need, dev, stream)
        nq = workspace.data_ptr()
    try:
        args = _pack_head_norm_backward(dq_out.data_ptr(), xq, xsq, wq, oq, dwq, kgq, kq, ksq, kwq, koq, kdwq, tc, ts, tp, nq,
                                        gp, xp, op, kgp, kp, kop, need, rows, hq, hk, dim, rot, table, dt, wt,
                                        OPT_HEADS_INTERLEAVED if interleaved else 0, eps)
    except _NOT_HELD as e:
        raise ValueError(f"opt_head_norm_backward: {e}") from None
    st = ready.head_norm_backward(args, ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_head_norm_backward")


def opt_head_norm_backward_workspace(rows: int, q_heads: int, k_heads: int, dim: int) -> int:
    return _check(lib().opt_head_norm_backward_workspace(rows, q_heads, k_heads, dim), "opt_head_norm_backward_workspace")


def opt_matmul(a, a_scales, b, b_scales, out, addend=None, stream=None, wait_drill=False):
    """out = a b^T (+ addend): a of m x k and b of n x k codes with their scales,
    out and addend float32 or bfloat16 of m x n; addend may be out."""
    ready = _ready or _get_ready()
    dtype = out.dtype
    dt = ready.dtypes.get(dtype)
    if dt is None:
        _refuse_dtype(out, "out")
    dev = _device(out, "out", ready)
    m, n, op = _matrix(out, "out")
    k = a.shape[-1]
    aq, asq, ap = _held(a, a_scales, "a", m, k, dev, ready)
    bq, bsq, bp = _held(b, b_scales, "b", n, k, dev, ready)
    dq, dp = (0, 0) if addend is None else _like(addend, "addend", m, n, dtype, dev)
    st = ready.matmul(_pack_matmul(aq, asq, bq, bsq, dq, out.data_ptr(), ap, bp, dp, op, m, n, k, dt,
                                   OPT_MATMUL_WAIT_DRILL if wait_drill else 0),
                      ready.stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        _check(st, "opt_matmul")


def opt_matmul_form(a, b):
    """How opt_matmul computes a b^T of these codes on the current device: (CTAs
    that share a tile, its columns, parts of the depth, whether the tile's rows are
    b's, most tiles per CTA or pair); zeros where no tiles are formed."""
    (m, k, ap), (n, kb, bp) = _matrix(a, "a"), _matrix(b, "b")
    if k != kb:
        raise ValueError(f"a and b: depths {k} and {kb}")
    form = (_i32 * 5)()
    _check(lib().opt_matmul_form(_pack_matmul(a.data_ptr(), 0, b.data_ptr(), 0, 0, 0, ap, bp, 0, 0, m, n, k, 0, 0), form),
           "opt_matmul_form")
    return tuple(form)


def opt_layer_status(stream=None) -> int:
    """Error flags of the layer kernels since the last call (0: all ran to completion)."""
    out = _i32()
    _check(lib().opt_layer_status(_c.byref(out), _stream_ptr(stream)), "opt_layer_status")
    return out.value
