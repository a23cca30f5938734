"""Microscaled 4-bit (MX4) tensors and layers: Python binding of ``monarch_mx4_*``.

    q = mx4_quantise(W)                    # weight (nblocks, out_blk, in_blk)
    q = mx4_quantise(X, nblocks=4)         # activations (rows, 4 * in_blk)
    V = mx4_dequantise(q, "bf16")          # the values the codes stand for, in the same layout
    Y = mx4_linear_fwd(X, Wq)              # W in MX4 and X as it is (serving), or an Mx4 X (training)
    dX, dW, dbias = mx4_linear_bwd(dY, Xq, Wq, bias=True)
    Y = mx4_fwd(X, Rq, Lq, shape)          # Monarch map with both factors in MX4

Every 32 values along the inner axis share a power-of-two scale and are held in 4 bits
(``include/monarch.h`` has the format).  Work runs on the tensors' device, on ``stream`` or that
device's current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import (MONARCH_BF16, MonarchDims, MonarchMx4Dims, MonarchMx4LinearDims, _check, _check_tensors, _require_cuda,
               _torch_dtype, dtype_code, lib)


class Mx4:
    """A quantised tensor: ``nblocks`` matrices of (rows, cols), scales shared along cols.

    ``codes`` and ``scales`` are contiguous uint8 CUDA tensors in the layout of ``include/monarch.h``;
    ``by_block`` says which plain layout it came from: (nblocks, rows, cols), or (rows, nblocks * cols);
    ``dtype`` is that tensor's type ("bf16" / "f32")."""

    __slots__ = ("codes", "scales", "rows", "nblocks", "cols", "by_block", "dtype")

    def __init__(self, codes, scales, rows: int, nblocks: int, cols: int, by_block: bool, dtype):
        self.rows, self.nblocks, self.cols, self.by_block = int(rows), int(nblocks), int(cols), bool(by_block)
        self.dtype = "bf16" if dtype_code(dtype) == MONARCH_BF16 else "f32"
        self.codes, self.scales = codes, scales
        need = _buffer_bytes(_dims(self, self.dtype))
        for name, t, n in (("codes", codes, need[0]), ("scales", scales, need[1])):
            if t.dtype != torch.uint8 or t.numel() != n:
                raise ValueError("%s must be uint8 with %d elements" % (name, n))

    @property
    def device(self):
        return self.codes.device

    @property
    def shape(self):
        """Shape of the plain tensor."""
        return (self.nblocks, self.rows, self.cols) if self.by_block else (self.rows, self.nblocks * self.cols)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def __repr__(self):
        return "Mx4(shape=%s, nblocks=%d, dtype=%s)" % (tuple(self.shape), self.nblocks, self.dtype)


def _dims(q, dtype) -> MonarchMx4Dims:
    return MonarchMx4Dims(q.rows, q.nblocks, q.cols, int(q.by_block), dtype_code(dtype))


def _buffer_bytes(d) -> tuple:
    """(codes, scales) bytes; raises MonarchError on sizes that the library does not take."""
    L, p = lib(), ctypes.byref(d)
    codes, scales = int(L.monarch_mx4_code_bytes(p)), int(L.monarch_mx4_scale_bytes(p))
    if codes == 0 and d.rows != 0:
        _check("monarch_mx4_quantise", L.monarch_mx4_quantise(None, p, None, None, None))
    return codes, scales


def _same_device(*ts):
    """Contiguous CUDA tensors of one device; returns it."""
    _require_cuda(*ts)
    device = None
    for t in ts:
        if t is not None:
            if device is None:
                device = t.device
            elif t.device != device:
                raise ValueError("tensors on %s and %s: one call takes one device's" % (device, t.device))
    return device


def _empty(shape, dtype, device, stream):
    """Memory for work on `stream` (None: the device's current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(name, device, stream, *args):
    """The C entry point `name` with args and the stream handle, `device` being the current one."""
    fn = getattr(lib(), name)
    s = ctypes.c_void_p((torch.cuda.current_stream(device) if stream is None else stream).cuda_stream)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    _check(name, rc)


def _p(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace, need, device, stream):
    """(tensor to keep alive, address, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty(need, torch.uint8, device, stream)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def mx4_quantise(X, nblocks: int | None = None, stream=None) -> Mx4:
    """X in MX4.  A 3-D X is a weight (nblocks, out_blk, in_blk); a 2-D X (rows, nblocks * cols) holds
    activations of `nblocks` blocks (default 1).  Scales never span two rows or two blocks."""
    code = dtype_code(X.dtype)
    if X.dim() == 3:
        nb, rows, cols = X.shape
        if nblocks is not None and nblocks != nb:
            raise ValueError("X has %d blocks, nblocks is %d" % (nb, nblocks))
    elif X.dim() == 2:
        nb = 1 if nblocks is None else int(nblocks)
        rows, width = X.shape
        if nb <= 0 or width % nb:
            raise ValueError("%d columns do not divide into %d blocks" % (width, nb))
        cols = width // nb
    else:
        raise ValueError("X must have 2 or 3 dimensions, got %d" % X.dim())
    device = _same_device(X)
    d = MonarchMx4Dims(rows, nb, cols, int(X.dim() == 3), code)
    nc, ns = _buffer_bytes(d)
    q = Mx4.__new__(Mx4)
    q.codes, q.scales = _empty(nc, torch.uint8, device, stream), _empty(ns, torch.uint8, device, stream)
    q.rows, q.nblocks, q.cols, q.by_block = rows, nb, cols, X.dim() == 3
    q.dtype = "bf16" if code == MONARCH_BF16 else "f32"
    _call("monarch_mx4_quantise", device, stream, _p(X), ctypes.byref(d), _p(q.codes), _p(q.scales))
    return q


def mx4_dequantise(q: Mx4, dtype=None, out=None, stream=None):
    """The values of q in the layout it came from, in `dtype` (default: the type it came in)."""
    code = dtype_code(q.dtype if dtype is None else dtype)
    dt = _torch_dtype(code)
    if out is None:
        out = _empty(q.shape, dt, q.device, stream)
    elif tuple(out.shape) != tuple(q.shape) or out.dtype != dt:
        raise ValueError("out must be %s of shape %s" % (dt, tuple(q.shape)))
    device = _same_device(q.codes, q.scales, out)
    _call("monarch_mx4_dequantise", device, stream, _p(q.codes), _p(q.scales), ctypes.byref(_dims(q, code)), _p(out))
    return out


def _weight(W, name="W"):
    if not isinstance(W, Mx4) or not W.by_block:
        raise ValueError("%s must be an Mx4 weight: mx4_quantise of (nblocks, out_blk, in_blk)" % name)


def _activations(X, W):
    if X.by_block or X.nblocks != W.nblocks or X.cols != W.cols:
        raise ValueError("X is %r, W %r: an Mx4 X must hold activations with W's blocks" % (X, W))


def _expect(dtype, **ts):
    for name, (t, shape) in ts.items():
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype):
            raise ValueError("%s must be %s of shape %s, is %s of shape %s" % (name, dtype, shape, t.dtype, tuple(t.shape)))


def mx4_linear_workspace_bytes(rows: int, nblocks: int, in_blk: int, out_blk: int, dtype="bf16", bias: bool = False,
                               backward: bool = False) -> int:
    """Workspace of mx4_linear_fwd with a plain X, or of mx4_linear_bwd."""
    d = MonarchMx4LinearDims(int(rows), int(nblocks), int(in_blk), int(out_blk), int(bool(bias)), dtype_code(dtype))
    f = lib().monarch_mx4_linear_bwd_workspace_bytes if backward else lib().monarch_mx4_linear_wfwd_workspace_bytes
    return int(f(ctypes.byref(d)))


def mx4_linear_fwd(X, W: Mx4, bias=None, Y=None, dtype=None, workspace=None, stream=None):
    """Block-diagonal linear layer with W in MX4: Y[r, b*out + o] = sum_i X[r, b*in + i] W[b, o, i] + bias.

    X is a plain tensor (rows, nblocks * in_blk), or an Mx4 of one; then Y has `dtype` (default: the type
    X was quantised from)."""
    _weight(W)
    both = isinstance(X, Mx4)
    if both:
        _activations(X, W)
        code = dtype_code(X.dtype if dtype is None else dtype)
        rows = X.rows
    else:
        code = dtype_code(X.dtype)
        if dtype is not None and dtype_code(dtype) != code:
            raise ValueError("dtype is X's unless X is an Mx4")
        rows = X.shape[0]
        _expect(X.dtype, X=(X, (rows, W.nblocks * W.cols)))
    dt = _torch_dtype(code)
    n_out = W.nblocks * W.rows
    _expect(dt, bias=(bias, (n_out,)), Y=(Y, (rows, n_out)))
    if Y is None:
        Y = _empty((rows, n_out), dt, W.device, stream)
    d = MonarchMx4LinearDims(rows, W.nblocks, W.cols, W.rows, int(bias is not None), code)
    if both:
        device = _same_device(X.codes, X.scales, W.codes, W.scales, bias, Y)
        _call("monarch_mx4_linear_fwd", device, stream, _p(X.codes), _p(X.scales), _p(W.codes), _p(W.scales), _p(bias),
              ctypes.byref(d), _p(Y))
    else:
        device = _same_device(X, W.codes, W.scales, bias, Y, workspace)
        need = int(lib().monarch_mx4_linear_wfwd_workspace_bytes(ctypes.byref(d)))
        workspace, wp, wn = _workspace(workspace, need, device, stream)
        _call("monarch_mx4_linear_wfwd", device, stream, _p(X), _p(W.codes), _p(W.scales), _p(bias), ctypes.byref(d), _p(Y),
              wp, wn)
    return Y


def mx4_linear_bwd(dY, X, W, bias: bool = False, need_dX: bool = True, dX=None, dW=None, dbias=None, workspace=None,
                   stream=None):
    """(dX, dW, dbias) of mx4_linear_fwd(X, W) for its quantised operands; a training step passes them on
    to the tensors X and W were rounded from.  X = None (a frozen layer) leaves out dW; need_dX = False
    leaves out dX; dbias is None without `bias`."""
    _weight(W)
    code = dtype_code(dY.dtype)
    rows = dY.shape[0]
    n_in, n_out = W.nblocks * W.cols, W.nblocks * W.rows
    if X is not None:
        if not isinstance(X, Mx4):
            raise ValueError("X must be the forward's Mx4 X, or None")
        _activations(X, W)
        if X.rows != rows:
            raise ValueError("X has %d rows, dY %d" % (X.rows, rows))
    elif dW is not None:
        raise ValueError("dW needs X")
    _expect(dY.dtype, dY=(dY, (rows, n_out)), dX=(dX, (rows, n_in)), dW=(dW, (W.nblocks, W.rows, W.cols)),
            dbias=(dbias, (n_out,)))
    device = _same_device(dY, W.codes, W.scales, dX, dW, dbias, workspace, *((X.codes, X.scales) if X is not None else ()))
    if need_dX and dX is None:
        dX = _empty((rows, n_in), dY.dtype, device, stream)
    if X is not None and dW is None:
        dW = _empty((W.nblocks, W.rows, W.cols), dY.dtype, device, stream)
    if bias and dbias is None:
        dbias = _empty((n_out,), dY.dtype, device, stream)
    d = MonarchMx4LinearDims(rows, W.nblocks, W.cols, W.rows, int(bool(bias)), code)
    need = int(lib().monarch_mx4_linear_bwd_workspace_bytes(ctypes.byref(d)))
    workspace, wp, wn = _workspace(workspace, need, device, stream)
    _call("monarch_mx4_linear_bwd", device, stream, _p(dY), _p(X.codes) if X is not None else None,
          _p(X.scales) if X is not None else None, _p(W.codes), _p(W.scales), ctypes.byref(d),
          _p(dX) if need_dX else None, _p(dW), _p(dbias) if bias else None, wp, wn)
    return dX if need_dX else None, dW, dbias if bias else None


def mx4_fwd(X, R: Mx4, L: Mx4, shape: dict, Y=None, workspace=None, stream=None):
    """Monarch map Y = X M^T with both factors in MX4 (fwd() with the factors' quantised values)."""
    _weight(R, "R")
    _weight(L, "L")
    for name, q, want in (("R", R, (shape["nb1"], shape["out1"], shape["in1"])),
                          ("L", L, (shape["nb2"], shape["out2"], shape["in2"]))):
        if tuple(q.shape) != tuple(want):
            raise ValueError("%s has shape %s, the dims need %s" % (name, tuple(q.shape), tuple(want)))
    code = dtype_code(X.dtype)
    rows = X.shape[0]
    _check_tensors(shape, rows, X.dtype, X=X, Y=Y)
    if Y is None:
        Y = _empty((rows, shape["nb2"] * shape["out2"]), X.dtype, X.device, stream)
    d = MonarchDims(rows, shape["nb1"], shape["in1"], shape["out1"], shape["nb2"], shape["in2"], shape["out2"],
                    int(shape.get("out_transpose", 1)), code)
    device = _same_device(X, R.codes, R.scales, L.codes, L.scales, Y, workspace)
    need = int(lib().monarch_mx4_fwd_workspace_bytes(ctypes.byref(d)))
    workspace, wp, wn = _workspace(workspace, need, device, stream)
    _call("monarch_mx4_fwd", device, stream, _p(X), _p(R.codes), _p(R.scales), _p(L.codes), _p(L.scales), ctypes.byref(d),
          _p(Y), wp, wn)
    return Y
