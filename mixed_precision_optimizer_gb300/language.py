"""Language-model operators of ``libmpopt.so``: what stands before, between and
behind the feed-forward blocks when they train on tokens.

* ``embedding``                 -- rows of a table by token, scaled
* ``embedding_backward``        -- their gradient, into the table's fp32 main_grad
* ``gated_recurrence``          -- h_t = h_{t-1} + sigmoid(gate_t) (x_t - h_{t-1})
  along the rows of packed sequences, or one token of each
* ``gated_recurrence_backward`` -- its gradients
* ``checkpoint_save``           -- an activation in e4m3, a power of two to every
  32 columns
* ``checkpoint_restore``        -- the activation back, through its activation
  function, and the gradient passing that
* ``cross_entropy``             -- loss and log-sum-exp of rows of logits, and the
  logits' gradient

Buffers, streams, devices and errors are as in ``feedforward``: the caller owns
every buffer, outputs are written in place on the current CUDA stream or on
``stream``, matrices have contiguous rows that may be slices of wider ones,
arguments that the library refuses raise ``MpoptError``, tensors of a wrong
type, device or shape ``TypeError`` or ``ValueError``.  Tokens and labels are
int32 or int64.  ``include/mpopt.h`` defines every operator.
"""

from __future__ import annotations

import ctypes
import struct

import mixed_precision_optimizer_gb300 as mp
from . import feedforward as ff
from .feedforward import ACTIVATIONS, _code, _elsewhere, _FLOAT, _lead, _mat, _stream, _vec, _workspace

_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

INDEX_INT32, INDEX_INT64 = 0, 1
CHECKPOINT_BLOCK = 32
STATE_ROWS = 8                # opt_recurrence_state_rows
MAIL_SELFTEST_THREADS = 64


class OptEmbeddingArgs(ctypes.Structure):
    _fields_ = [("tokens", _vp), ("table", _vp), ("y", _vp), ("rows", _i64), ("vocab", _i64), ("cols", _i64),
                ("table_ld", _i64), ("y_ld", _i64), ("index_dtype", _i32), ("dtype", _i32), ("y_dtype", _i32),
                ("scale", _f32)]


class OptEmbeddingGradArgs(ctypes.Structure):
    _fields_ = [("tokens", _vp), ("dy", _vp), ("dtable", _vp), ("rows", _i64), ("vocab", _i64), ("cols", _i64),
                ("dy_ld", _i64), ("index_dtype", _i32), ("dtype", _i32), ("accumulate", _i32), ("scale", _f32)]


class OptRecurrenceArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("gate", _vp), ("starts", _vp), ("h0", _vp), ("y", _vp), ("hT", _vp), ("states", _vp),
                ("rows", _i64), ("cols", _i64), ("sequences", _i64), ("x_ld", _i64), ("gate_ld", _i64), ("y_ld", _i64),
                ("dtype", _i32), ("reserved", _i32)]


class OptRecurrenceGradArgs(ctypes.Structure):
    _fields_ = [("dy", _vp), ("x", _vp), ("gate", _vp), ("starts", _vp), ("h0", _vp), ("states", _vp), ("dhT", _vp),
                ("dx", _vp), ("dgate", _vp), ("dh0", _vp), ("rows", _i64), ("cols", _i64), ("sequences", _i64),
                ("dy_ld", _i64), ("x_ld", _i64), ("gate_ld", _i64), ("dx_ld", _i64), ("dgate_ld", _i64),
                ("dtype", _i32), ("reserved", _i32)]


class OptCheckpointArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("scale", _vp), ("dy", _vp), ("z", _vp), ("y", _vp), ("dz", _vp), ("rows", _i64),
                ("cols", _i64), ("q_ld", _i64), ("scale_ld", _i64), ("dy_ld", _i64), ("z_ld", _i64), ("y_ld", _i64),
                ("dz_ld", _i64), ("act", _i32), ("reserved", _i32)]


class OptCrossEntropyArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("labels", _vp), ("weight", _vp), ("loss", _vp), ("lse", _vp), ("dlogits", _vp),
                ("rows", _i64), ("cols", _i64), ("logits_ld", _i64), ("dlogits_ld", _i64), ("dtype", _i32),
                ("index_dtype", _i32), ("scale", _f32), ("reserved", _i32)]


def declare(L):
    """Argument types of this module's entry points (see feedforward.declare)."""
    for name, args, res in (
            ("opt_embedding_forward", [_vp, _vp], ctypes.c_int),
            ("opt_embedding_backward", [_vp, _vp, _sz, _vp], ctypes.c_int),
            ("opt_embedding_workspace_size", [_i64, _i64, _i64], _sz),
            ("opt_recurrence_forward", [_vp, _vp], ctypes.c_int),
            ("opt_recurrence_backward", [_vp, _vp], ctypes.c_int),
            ("opt_recurrence_state_rows", [_i32], _i64),
            ("opt_checkpoint_save", [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
            ("opt_checkpoint_restore", [_vp, _vp], ctypes.c_int),
            ("opt_cross_entropy", [_vp, _vp], ctypes.c_int),
            ("opt_selftest_mail", [_vp, _i32, _i32, _i32, _vp], ctypes.c_int)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


_PACK_EMBEDDING = struct.Struct("=3Q5q3if").pack
_PACK_EMBEDDING_GRAD = struct.Struct("=3Q4q3if").pack
_PACK_RECURRENCE = struct.Struct("=7Q6q2i").pack
_PACK_RECURRENCE_GRAD = struct.Struct("=10Q8q2i").pack
_PACK_CHECKPOINT = struct.Struct("=6Q8q2i").pack
_PACK_CROSS_ENTROPY = struct.Struct("=6Q4q2ifi").pack


# --------------------------------------------------------------------------
# marshalling
# --------------------------------------------------------------------------

_torch = None
_INDEX = {}                   # torch dtype -> OPT_INDEX_*


def _load_torch():
    global _torch
    torch = ff._torch or ff._load_torch()
    _INDEX.update({torch.int32: INDEX_INT32, torch.int64: INDEX_INT64})
    _torch = torch
    return torch


def _indices(t, n, what, dev):
    """(pointer, OPT_INDEX_*) of a dense array of n tokens or labels."""
    code = _INDEX.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be int32 or int64, got {t.dtype}")
    if t.get_device() != dev:
        _elsewhere(t, dev, what)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} elements")
    return t.data_ptr(), code


def _grid(t, rows, cols, what, dev):
    """Pointer of a dense fp32 matrix argument; 0 for None."""
    if t is not None and t.shape != (rows, cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    return _vec(t, _torch.float32, rows * cols, what, dev)


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embedding(tokens, table, y, scale=1.0, stream=None):
    """y [rows][cols] = table[token] * scale for tokens [rows] (any shape, int32
    or int64); table [vocab][cols] and y are bf16 or fp32, each of its own type.
    A token outside [0, vocab) gives a row of zeros."""
    _torch or _load_torch()
    code, ycode = _code(table, "table", _FLOAT), _code(y, "y", _FLOAT)
    dev, vocab, cols, tp, tl = _lead(table, "table")
    rows = tokens.numel()
    ip, icode = _indices(tokens, rows, "tokens", dev)
    yp, yl = _mat(y, y.dtype, rows, cols, "y", dev)
    a = _PACK_EMBEDDING(ip, tp, yp, rows, vocab, cols, tl, yl, icode, code, ycode, scale)
    status = mp.lib().opt_embedding_forward(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_embedding_forward")


def embedding_backward(tokens, dy, dtable, scale=1.0, accumulate=True, workspace=None, stream=None):
    """dtable [vocab][cols] (fp32 main_grad) += scale * the sums of dy's rows
    (bf16 or fp32) that belong to each token; accumulate=False overwrites all of
    dtable.  Tokens outside [0, vocab) add nothing.  Needs
    embedding_workspace(rows, vocab, cols)."""
    _torch or _load_torch()
    code = _code(dy, "dy", _FLOAT)
    dev, rows, cols, yp, yl = _lead(dy, "dy")
    ip, icode = _indices(tokens, rows, "tokens", dev)
    if len(dtable.shape) != 2 or dtable.shape[1] != cols:
        raise ValueError(f"dtable has shape {tuple(dtable.shape)}, expected (vocab, {cols})")
    vocab = dtable.shape[0]
    gp = _vec(dtable, _torch.float32, vocab * cols, "dtable", dev)
    a = _PACK_EMBEDDING_GRAD(ip, yp, gp, rows, vocab, cols, yl, icode, code, 1 if accumulate else 0, scale)
    ws, nb = _workspace(workspace, dev)
    status = mp.lib().opt_embedding_backward(a, ws, nb, _stream(stream, dev))
    if status:
        mp._check(status, "opt_embedding_backward")


def embedding_workspace_size(rows, vocab, cols) -> int:
    return int(mp.lib().opt_embedding_workspace_size(int(rows), int(vocab), int(cols)))


def embedding_workspace(rows, vocab, cols, device=None):
    """Workspace of embedding_backward for up to this many rows, tokens and columns."""
    return mp.alloc_workspace(embedding_workspace_size(rows, vocab, cols), device)


# --------------------------------------------------------------------------
# gated recurrence
# --------------------------------------------------------------------------

def recurrence_states(rows, cols, dtype, device=None):
    """Buffer for gated_recurrence's states: what gated_recurrence_backward needs
    of a forward pass over this many rows of this type (bf16 or fp32).  Only that
    reads it; where it has no use for a value, the forward pass writes none."""
    torch = _torch or _load_torch()
    if ff._CODES.get(dtype) not in _FLOAT:
        raise TypeError(f"unsupported type, {dtype}")
    return torch.empty((-(-int(rows) // STATE_ROWS), int(cols)), dtype=torch.float32, device=device or "cuda")


def _states(t, rows, cols, dev):
    return _grid(t, -(-rows // STATE_ROWS), cols, "states", dev)


def _sequences(starts, sequences):
    """The number of sequences, by default that of starts, or one."""
    if sequences is None:
        sequences = 1 if starts is None else starts.numel() - 1
    if starts is not None and starts.numel() != sequences + 1:
        raise ValueError(f"starts has {starts.numel()} elements, expected {sequences + 1}")
    return sequences


def gated_recurrence(x, gate, y, starts=None, sequences=None, h0=None, hT=None, states=None, stream=None):
    """For every column by itself, along the rows of each sequence:
    h_t = h_{t-1} + sigmoid(gate_t) (x_t - h_{t-1}), y_t = h_t, from h0
    [sequences][cols] (fp32; None: zeros) to hT.  x, gate and y are bf16 or fp32,
    all of one type; h is fp32.  The sequences' rows are packed: sequence s has
    rows starts[s] .. starts[s + 1] - 1 (int32 [sequences + 1]), or, with starts
    None, all have rows / sequences (one sequence by default).  With one row to a
    sequence and no starts hT may be h0 itself.  states (recurrence_states) keeps
    what the gradient needs."""
    torch = _torch or _load_torch()
    code, dt = _code(x, "x", _FLOAT), x.dtype
    dev, rows, cols, xp, xl = _lead(x, "x")
    gp, gl = _mat(gate, dt, rows, cols, "gate", dev)
    yp, yl = _mat(y, dt, rows, cols, "y", dev)
    sequences = _sequences(starts, sequences)
    sp = _vec(starts, torch.int32, sequences + 1, "starts", dev)
    a = _PACK_RECURRENCE(xp, gp, sp, _grid(h0, sequences, cols, "h0", dev), yp, _grid(hT, sequences, cols, "hT", dev),
                         _states(states, rows, cols, dev), rows, cols, sequences, xl, gl, yl, code, 0)
    status = mp.lib().opt_recurrence_forward(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_recurrence_forward")


def gated_recurrence_backward(dy, x, gate, states, dx, dgate, starts=None, sequences=None, h0=None, dhT=None, dh0=None,
                              stream=None):
    """Gradients of gated_recurrence with respect to x, gate and h0 (dh0, fp32
    [sequences][cols], optional) from dy and dhT (fp32, None: zeros).  x, gate,
    starts and h0 are the forward call's, states what it wrote."""
    torch = _torch or _load_torch()
    code, dt = _code(x, "x", _FLOAT), x.dtype
    dev, rows, cols, xp, xl = _lead(x, "x")
    yp, yl = _mat(dy, dt, rows, cols, "dy", dev)
    gp, gl = _mat(gate, dt, rows, cols, "gate", dev)
    dxp, dxl = _mat(dx, dt, rows, cols, "dx", dev)
    dgp, dgl = _mat(dgate, dt, rows, cols, "dgate", dev)
    sequences = _sequences(starts, sequences)
    sp = _vec(starts, torch.int32, sequences + 1, "starts", dev)
    a = _PACK_RECURRENCE_GRAD(yp, xp, gp, sp, _grid(h0, sequences, cols, "h0", dev), _states(states, rows, cols, dev),
                              _grid(dhT, sequences, cols, "dhT", dev), dxp, dgp, _grid(dh0, sequences, cols, "dh0", dev),
                              rows, cols, sequences, yl, xl, gl, dxl, dgl, code, 0)
    status = mp.lib().opt_recurrence_backward(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_recurrence_backward")


# --------------------------------------------------------------------------
# checkpoints in 8 bits
# --------------------------------------------------------------------------

def checkpoint_save(x, q, scale, stream=None):
    """q [rows][cols] (float8_e4m3fn), scale [rows][ceil(cols / 32)] (uint8) <- x
    (bf16 or fp32): x ~ q * 2^(scale - 127), a power of two to every 32 columns of
    a row."""
    torch = _torch or _load_torch()
    code = _code(x, "x", _FLOAT)
    dev, rows, cols, xp, xl = _lead(x, "x")
    qp, ql = _mat(q, torch.float8_e4m3fn, rows, cols, "q", dev)
    sp, sl = _mat(scale, torch.uint8, rows, -(-cols // CHECKPOINT_BLOCK), "scale", dev)
    status = mp.lib().opt_checkpoint_save(xp, xl, code, rows, cols, qp, ql, sp, sl, _stream(stream, dev))
    if status:
        mp._check(status, "opt_checkpoint_save")


def checkpoint_restore(q, scale, z=None, y=None, act="none", dy=None, dz=None, stream=None):
    """From a checkpoint z = q * 2^(scale - 127), all bf16 and optional: z itself
    (exact), y = act(z), and dz = dy * act'(z) (which may be dy itself)."""
    torch = _torch or _load_torch()
    acode = ACTIVATIONS.get(act)
    if acode is None:
        raise ValueError(f"unknown activation {act!r}")
    bf16 = torch.bfloat16
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"q must be {torch.float8_e4m3fn}, got {q.dtype}")
    dev, rows, cols, qp, ql = _lead(q, "q")
    sp, sl = _mat(scale, torch.uint8, rows, -(-cols // CHECKPOINT_BLOCK), "scale", dev)
    dyp, dyl = _mat(dy, bf16, rows, cols, "dy", dev)
    zp, zl = _mat(z, bf16, rows, cols, "z", dev)
    yp, yl = _mat(y, bf16, rows, cols, "y", dev)
    dzp, dzl = _mat(dz, bf16, rows, cols, "dz", dev)
    a = _PACK_CHECKPOINT(qp, sp, dyp, zp, yp, dzp, rows, cols, ql, sl, dyl, zl, yl, dzl, acode, 0)
    status = mp.lib().opt_checkpoint_restore(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_checkpoint_restore")


# --------------------------------------------------------------------------
# cross-entropy
# --------------------------------------------------------------------------

def cross_entropy(logits, labels, loss=None, lse=None, dlogits=None, scale=1.0, weight=None, stream=None):
    """loss [rows] (fp32) = lse - logits_label with lse = log sum exp(logits) for
    rows of logits (bf16 or fp32); dlogits (of their type, may be logits itself) =
    (softmax(logits) - onehot(label)) * scale * weight, weight [rows] fp32 or
    None.  A label outside [0, cols) is ignored: loss 0, dlogits 0."""
    torch = _torch or _load_torch()
    code, f32 = _code(logits, "logits", _FLOAT), torch.float32
    dev, rows, cols, xp, xl = _lead(logits, "logits")
    lp, icode = _indices(labels, rows, "labels", dev)
    gp, gl = _mat(dlogits, logits.dtype, rows, cols, "dlogits", dev)
    a = _PACK_CROSS_ENTROPY(xp, lp, _vec(weight, f32, rows, "weight", dev), _vec(loss, f32, rows, "loss", dev),
                            _vec(lse, f32, rows, "lse", dev), gp, rows, cols, xl, gl, code, icode, scale, 0)
    status = mp.lib().opt_cross_entropy(a, _stream(stream, dev))
    if status:
        mp._check(status, "opt_cross_entropy")


# --------------------------------------------------------------------------
# self-test
# --------------------------------------------------------------------------

def selftest_mail(sums, held_back=-1, stream=None):
    """The messages between the CTAs of a cluster, with a part of one held back (see
    opt_selftest_mail).  sums [CTAs][messages][64] fp32: what each thread received,
    NaN for a message that did not come.  For tests of the failure path."""
    torch = _torch or _load_torch()
    ctas, messages, threads = sums.shape
    if threads != MAIL_SELFTEST_THREADS:
        raise ValueError(f"sums has shape {tuple(sums.shape)}, expected (CTAs, messages, {MAIL_SELFTEST_THREADS})")
    dev = _lead(sums, "sums")[0]
    status = mp.lib().opt_selftest_mail(_vec(sums, torch.float32, sums.numel(), "sums", dev), ctas, messages, held_back,
                                        _stream(stream, dev))
    if status:
        mp._check(status, "opt_selftest_mail")
