"""Feed-forward operators of ``libmpopt.so``: the layers around the parameters.

The bf16 model copies that the optimizer step writes are the weights here, and
the fp32 ``main_grad`` buffers that it reads are the outputs:

* ``rmsnorm``           -- h = x + residual, y = rmsnorm(h) * gamma in bf16
  and / or in e4m3 with a scale per row
* ``rmsnorm_backward``  -- its gradient; dgamma into fp32 main_grad
* ``quantize_rows``     -- a matrix in e4m3 with a scale per row
* ``linear``            -- y = act(x w^T + bias) + residual, bf16 or e4m3 operands
* ``linear_backward``   -- dx, and dw and dbias into fp32 main_grad

As in the rest of the package the caller owns every buffer: outputs are
passed in and written in place, on the current CUDA stream or on ``stream``.
Matrices are 2-D (or more leading dimensions that collapse into rows without a
copy; a vector is one row) with contiguous rows that may be slices of wider
ones.  All tensors and the workspace are on the current device.
``include/mpopt.h`` defines every operator; arguments it refuses raise
``MpoptError``, tensors of a wrong type, device or shape ``TypeError`` or
``ValueError``.
"""

from __future__ import annotations

import ctypes
import struct

import mixed_precision_optimizer_gb300 as mp

_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

DTYPE_FP32, DTYPE_BF16, DTYPE_E4M3 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
LINEAR_ANY_LAYOUT = 1
LINEAR_HEADER_BYTES = 256


class OptRmsnormArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("gamma", _vp), ("h", _vp), ("y", _vp), ("q", _vp), ("q_scale", _vp),
                ("rstd", _vp), ("rows", _i64), ("cols", _i64), ("x_ld", _i64), ("residual_ld", _i64), ("h_ld", _i64),
                ("y_ld", _i64), ("q_ld", _i64), ("dtype", _i32), ("gamma_dtype", _i32), ("eps", _f32),
                ("reserved", _i32)]


class OptRmsnormGradArgs(ctypes.Structure):
    _fields_ = [("dy", _vp), ("h", _vp), ("gamma", _vp), ("rstd", _vp), ("dh", _vp), ("dx", _vp), ("dgamma", _vp),
                ("rows", _i64), ("cols", _i64), ("dy_ld", _i64), ("h_ld", _i64), ("dh_ld", _i64), ("dx_ld", _i64),
                ("dtype", _i32), ("gamma_dtype", _i32), ("accumulate", _i32), ("reserved", _i32)]


class OptLinearArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("w", _vp), ("x_scale", _vp), ("w_scale", _vp), ("bias", _vp), ("residual", _vp),
                ("y", _vp), ("z", _vp), ("m", _i64), ("n", _i64), ("k", _i64), ("x_ld", _i64), ("w_ld", _i64),
                ("residual_ld", _i64), ("y_ld", _i64), ("z_ld", _i64), ("dtype", _i32), ("bias_dtype", _i32),
                ("act", _i32), ("reserved", _i32)]


class OptLinearGradArgs(ctypes.Structure):
    _fields_ = [("dz", _vp), ("x", _vp), ("w", _vp), ("z_prev", _vp), ("dx", _vp), ("dw", _vp), ("dbias", _vp),
                ("m", _i64), ("n", _i64), ("k", _i64), ("dz_ld", _i64), ("x_ld", _i64), ("w_ld", _i64),
                ("z_prev_ld", _i64), ("dx_ld", _i64), ("act_prev", _i32), ("accumulate", _i32)]


def declare(L):
    """Argument types of this module's entry points.  Argument structs are
    passed as c_void_p: a ctypes struct (by reference) or, from the functions
    below, its packed bytes."""
    for name, args, res in (
            ("opt_rmsnorm_forward", [_vp, _vp], ctypes.c_int),
            ("opt_rmsnorm_backward", [_vp, _vp, _sz, _vp], ctypes.c_int),
            ("opt_rmsnorm_workspace_size", [_i64, _i64], _sz),
            ("opt_quantize_rows", [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _vp], ctypes.c_int),
            ("opt_linear_forward", [_vp, _vp, _sz, _vp], ctypes.c_int),
            ("opt_linear_backward", [_vp, _vp, _sz, _vp], ctypes.c_int),
            ("opt_linear_workspace_size", [_i64, _i64, _i64, _i32], _sz)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# The calls below are short enough for their host time to show (a norm of one
# token takes 2 us on the GPU), so they pack the argument structs with one
# struct.pack (0.6 us, a ctypes constructor 2 us) and read the current stream's
# handle directly (0.1 us, torch.cuda.current_stream() 3 us).
_PACK_NORM = struct.Struct("=8Q7q2ifi").pack
_PACK_NORM_GRAD = struct.Struct("=7Q6q4i").pack
_PACK_LINEAR = struct.Struct("=8Q8q4i").pack
_PACK_LINEAR_GRAD = struct.Struct("=7Q8q2i").pack


# --------------------------------------------------------------------------
# marshalling
# --------------------------------------------------------------------------

_torch = None                 # torch, once a call has needed it (importing this package does not load it)
_CODES = {}                   # torch dtype -> OPT_DTYPE_*
_raw_stream = None
_current_device = None        # torch's, without its checks (0.1 us)


def _load_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _CODES.update({torch.float32: DTYPE_FP32, torch.bfloat16: DTYPE_BF16, torch.float8_e4m3fn: DTYPE_E4M3})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch
    return torch


def _stream(stream, dev):
    """Handle of `stream`, by default the device's current stream."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _raw_stream is not None:
        return _raw_stream(dev)
    return _torch.cuda.current_stream(dev).cuda_stream


def _code(t, what, allowed):
    code = _CODES.get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{what} has an unsupported type, {t.dtype}")
    return code


_FLOAT = (DTYPE_FP32, DTYPE_BF16)


def _shape2(t, what):
    """(rows, cols) of a matrix argument; leading dimensions are rows."""
    shape = t.shape
    if len(shape) == 2:
        return shape
    if not shape:
        raise ValueError(f"{what} must have at least one dimension")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    return rows, shape[-1]


def _lead(t, what):
    """(device, rows, cols, pointer, distance between rows) of the matrix that
    sets a call's sizes and device.  That has to be the current device: the
    library launches there, whatever its arguments' addresses."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{what} is on cuda:{dev}, which is not the current device (cuda:{_current_device()})")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        t = t.view(_shape2(t, what))          # raises when the rows are not evenly spaced
        shape, stride = t.shape, t.stride()
    rows, cols = shape
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return dev, rows, cols, t.data_ptr(), stride[0]


def _elsewhere(t, dev, what):
    """Raises for a tensor that is not on the call's device."""
    if t.get_device() < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the other tensors on cuda:{dev}")


def _mat(t, dtype, rows, cols, what, dev):
    """(pointer, distance between rows) of a matrix argument; (0, 0) for None."""
    if t is None:
        return 0, 0
    stride = t.stride()
    if t.dtype is dtype and t.get_device() == dev and t.shape == (rows, cols) and stride[1] == 1:
        return t.data_ptr(), stride[0]
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    _elsewhere(t, dev, what)
    if len(stride) != 2:
        t = t.view(_shape2(t, what))          # raises when the rows are not evenly spaced
        stride = t.stride()
    if t.shape != (rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), stride[0]


def _vec(t, dtype, n, what, dev):
    """Pointer of a dense vector argument; 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    _elsewhere(t, dev, what)
    raise ValueError(f"{what} must be contiguous with {n} elements")


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev:
        _elsewhere(ws, dev, "workspace")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# --------------------------------------------------------------------------
# RMS norm and 8-bit rows
# --------------------------------------------------------------------------

def rmsnorm(x, gamma, eps=1e-6, residual=None, h=None, y=None, q=None, q_scale=None, rstd=None, stream=None):
    """h = x + residual (x and residual bf16 or fp32, h of their type);
    y = h / sqrt(mean(h^2) + eps) * gamma per row, written as bf16 (y), as
    e4m3 with fp32 row scales (q, q_scale), or both; rstd [rows] fp32 is what
    rmsnorm_backward needs.  Outputs left out are not written.  h may be x or
    residual itself."""
    torch = _torch or _load_torch()
    code, gcode = _code(x, "x", _FLOAT), _code(gamma, "gamma", _FLOAT)
    dt, f32 = x.dtype, torch.float32
    dev, rows, cols, xp, xl = _lead(x, "x")
    rp, rl = _mat(residual, dt, rows, cols, "residual", dev)
    hp, hl = _mat(h, dt, rows, cols, "h", dev)
    yp, yl = _mat(y, torch.bfloat16, rows, cols, "y", dev)
    qp, ql = _mat(q, torch.float8_e4m3fn, rows, cols, "q", dev)
    gp, sp = _vec(gamma, gamma.dtype, cols, "gamma", dev), _vec(q_scale, f32, rows, "q_scale", dev)
    a = _PACK_NORM(xp, rp, gp, hp, yp, qp, sp, _vec(rstd, f32, rows, "rstd", dev), rows, cols, xl, rl, hl, yl, ql, code,
                   gcode, eps, 0)
    status = mp.lib().opt_rmsnorm_forward(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_rmsnorm_forward")


def rmsnorm_backward(dy, h, gamma, rstd, dx, dh=None, dgamma=None, accumulate=True, workspace=None, stream=None):
    """Gradient of rmsnorm at h (its output, or x without a residual): dy bf16;
    dx (of h's type) is the gradient of x and of the residual, dh (optional)
    the gradient reaching h past the norm; dgamma fp32 [cols] is added to, or
    overwritten with accumulate=False, and needs rmsnorm_workspace(rows, cols)."""
    torch = _torch or _load_torch()
    code, gcode = _code(h, "h", _FLOAT), _code(gamma, "gamma", _FLOAT)
    f32 = torch.float32
    dev, rows, cols, hp, hl = _lead(h, "h")
    yp, yl = _mat(dy, torch.bfloat16, rows, cols, "dy", dev)
    sp, sl = _mat(dh, h.dtype, rows, cols, "dh", dev)
    xp, xl = _mat(dx, h.dtype, rows, cols, "dx", dev)
    gp, rp = _vec(gamma, gamma.dtype, cols, "gamma", dev), _vec(rstd, f32, rows, "rstd", dev)
    a = _PACK_NORM_GRAD(yp, hp, gp, rp, sp, xp, _vec(dgamma, f32, cols, "dgamma", dev), rows, cols, yl, hl, sl, xl, code,
                        gcode, 1 if accumulate else 0, 0)
    w, nb = _workspace(workspace, dev)
    status = mp.lib().opt_rmsnorm_backward(a, w, nb, _stream(stream, dev))
    if status:
        mp._check(status, "opt_rmsnorm_backward")


def rmsnorm_workspace_size(rows, cols) -> int:
    return int(mp.lib().opt_rmsnorm_workspace_size(int(rows), int(cols)))


def rmsnorm_workspace(rows, cols, device=None):
    """Workspace of rmsnorm_backward for up to this many rows and columns."""
    return mp.alloc_workspace(rmsnorm_workspace_size(rows, cols), device)


def quantize_rows(x, q, scale, stream=None):
    """q [rows][cols] (float8_e4m3fn), scale [rows] (fp32) <- x (bf16 or
    fp32): x ~ q * scale with the largest magnitude of a row at 448."""
    torch = _torch or _load_torch()
    code = _code(x, "x", _FLOAT)
    dev, rows, cols, xp, xl = _lead(x, "x")
    qp, ql = _mat(q, torch.float8_e4m3fn, rows, cols, "q", dev)
    sp = _vec(scale, torch.float32, rows, "scale", dev)
    status = mp.lib().opt_quantize_rows(xp, xl, code, rows, cols, qp, ql, sp, _stream(stream, dev))
    if status:
        mp._check(status, "opt_quantize_rows")


# --------------------------------------------------------------------------
# linear layer
# --------------------------------------------------------------------------

def linear_workspace_size(m, n, k, any_layout=False) -> int:
    """Workspace bytes of linear and linear_backward for x [m][k], w [n][k];
    any_layout: also for operands whose rows do not start on 16 bytes although
    dense ones of these sizes would.  The first LINEAR_HEADER_BYTES have to be
    zero before the first call; linear_workspace sees to that."""
    return int(mp.lib().opt_linear_workspace_size(int(m), int(n), int(k), LINEAR_ANY_LAYOUT if any_layout else 0))


def linear_workspace(m, n, k, any_layout=False, device=None):
    """A workspace of linear_workspace_size bytes with its header zeroed.  In
    stream order it serves any number of calls: of these sizes, and of smaller
    m, n and k -- with any_layout all of them, without it those whose operands'
    rows start on 16 bytes (dense rows of a multiple of 8 bf16 or 16 e4m3
    elements).  A call that needs more raises MpoptError."""
    ws = mp.alloc_workspace(linear_workspace_size(m, n, k, any_layout), device)
    if ws is not None:
        ws[:LINEAR_HEADER_BYTES].zero_()
    return ws


def linear(x, w, y, bias=None, act="none", residual=None, z=None, x_scale=None, w_scale=None, workspace=None,
           stream=None):
    """y [m][n] = act(x w^T + bias) + residual (bf16).  x [m][k] and w [n][k]
    are bf16, or float8_e4m3fn with x_scale [m] and w_scale [n]; bias [n] is
    bf16 or fp32; z [m][n] (bf16, optional) receives the pre-activation.  y may
    be residual itself.  act: "none", "relu", "gelu" (tanh form), "silu"."""
    torch = _torch or _load_torch()
    code = _code(x, "x", (DTYPE_BF16, DTYPE_E4M3))
    acode = ACTIVATIONS.get(act)
    if acode is None:
        raise ValueError(f"unknown activation {act!r}")
    bf16, f32 = torch.bfloat16, torch.float32
    dev, m, k, xp, xl = _lead(x, "x")
    n = _shape2(w, "w")[0]
    wp, wl = _mat(w, x.dtype, n, k, "w", dev)
    rp, rl = _mat(residual, bf16, m, n, "residual", dev)
    yp, yl = _mat(y, bf16, m, n, "y", dev)
    zp, zl = _mat(z, bf16, m, n, "z", dev)
    bp, bcode = 0, DTYPE_BF16
    if bias is not None:
        bp, bcode = _vec(bias, bias.dtype, n, "bias", dev), _code(bias, "bias", _FLOAT)
    xsp, wsp = _vec(x_scale, f32, m, "x_scale", dev), _vec(w_scale, f32, n, "w_scale", dev)
    a = _PACK_LINEAR(xp, wp, xsp, wsp, bp, rp, yp, zp, m, n, k, xl, wl, rl, yl, zl, code, bcode, acode, 0)
    ws, nb = _workspace(workspace, dev)
    status = mp.lib().opt_linear_forward(a, ws, nb, _stream(stream, dev))
    if status:
        mp._check(status, "opt_linear_forward")


def linear_backward(dz, x, w, dx=None, z_prev=None, act_prev="none", dw=None, dbias=None, accumulate=True,
                    workspace=None, stream=None):
    """Gradients of z = x w^T + bias for dz [m][n] (bf16): dx [m][k] bf16 =
    (dz w) * act_prev'(z_prev) (with act_prev "none", which needs no z_prev,
    dz w); dw [n][k] and dbias [n] fp32 main_grad buffers, added to or
    overwritten (accumulate=False).
    Outputs left out are not computed; x and w may be None when only the other
    one's product is asked for."""
    torch = _torch or _load_torch()
    if x is None and w is None and dbias is None:
        raise ValueError("linear_backward: nothing to compute")
    k = _shape2(x, "x")[1] if x is not None else _shape2(w, "w")[1] if w is not None else 1
    acode = ACTIVATIONS.get(act_prev)
    if acode is None:
        raise ValueError(f"unknown activation {act_prev!r}")
    bf16, f32 = torch.bfloat16, torch.float32
    if dz.dtype != bf16:
        raise TypeError(f"dz must be {bf16}, got {dz.dtype}")
    dev, m, n, zp, zl = _lead(dz, "dz")
    xp, xl = _mat(x, bf16, m, k, "x", dev)
    wp, wl = _mat(w, bf16, n, k, "w", dev)
    pp, pl = _mat(z_prev, bf16, m, k, "z_prev", dev)
    dp, dl = _mat(dx, bf16, m, k, "dx", dev)
    if dw is not None and dw.shape != (n, k):
        raise ValueError(f"dw has shape {tuple(dw.shape)}, expected {(n, k)}")
    wgp, bgp = _vec(dw, f32, n * k, "dw", dev), _vec(dbias, f32, n, "dbias", dev)
    a = _PACK_LINEAR_GRAD(zp, xp, wp, pp, dp, wgp, bgp, m, n, k, zl, xl, wl, pl, dl, acode, 1 if accumulate else 0)
    ws, nb = _workspace(workspace, dev)
    status = mp.lib().opt_linear_backward(a, ws, nb, _stream(stream, dev))
    if status:
        mp._check(status, "opt_linear_backward")
