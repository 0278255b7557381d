"""Python binding of the training-layer operators (include/opt_layer.h):
dropout, residual RMS norm and its gradients, conversion to E4M3 with a scale
for each block of 128, and the product of two matrices held in that form.

Argument marshalling and shape checks only; the functions carry the C names
and write into tensors that the caller owns.  A matrix argument is a CUDA
tensor on the current device whose last dimension is contiguous: a 2-d tensor
of any row stride, or a contiguous tensor of any other shape, taken as rows of
its last dimension.  Wrong shapes and dtypes, and numbers that their C types do not
hold, raise ValueError; everything else is checked by the library (OptError).
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
    "opt_matmul": (_c.c_int, [_c.c_char_p, _vp]),
    "opt_matmul_form": (_c.c_int, [_c.c_char_p, _c.POINTER(_i32)]),
    "opt_layer_status": (_c.c_int, [_c.POINTER(_i32), _vp]),
}

OPT_MATMUL_WAIT_DRILL = 1

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
        self.f32 = torch.float32
        self.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        self.dropout, self.rms_norm, self.rms_norm_backward = L.opt_dropout, L.opt_rms_norm, L.opt_rms_norm_backward
        self.quantize, self.matmul = L.opt_quantize, L.opt_matmul


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
