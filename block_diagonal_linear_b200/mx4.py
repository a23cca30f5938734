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

from . import MONARCH_BF16, MONARCH_F32, MonarchDims, MonarchMx4Dims, MonarchMx4LinearDims, _check, dtype_code, lib

_DTYPES = {MONARCH_BF16: torch.bfloat16, MONARCH_F32: torch.float32}
_CODES = {torch.bfloat16: MONARCH_BF16, torch.float32: MONARCH_F32}
_byref = ctypes.byref
_raw_stream = torch._C._cuda_getCurrentRawStream  # address of a device's current stream
_current_device = torch._C._cuda_getDevice


class Mx4:
    """A quantised tensor: ``nblocks`` matrices of (rows, cols), scales shared along cols.

    ``codes`` and ``scales`` are contiguous uint8 CUDA tensors in the layout of ``include/monarch.h``;
    ``by_block`` says which plain layout it came from: (nblocks, rows, cols), or (rows, nblocks * cols);
    ``dtype`` is that tensor's type ("bf16" / "f32")."""

    # _hold: what keeps the memory alive; _pc, _ps: addresses of codes and scales; _index: their device;
    # _layers: dims of a layer or map with this weight and its workspace bytes, by the rest of the dims
    __slots__ = ("rows", "nblocks", "cols", "by_block", "code", "_hold", "_sizes", "_pc", "_ps", "_index", "_layers")

    def __init__(self, codes, scales, rows: int, nblocks: int, cols: int, by_block: bool, dtype):
        self._shape(int(rows), int(nblocks), int(cols), bool(by_block), dtype_code(dtype))
        for name, t, n in (("codes", codes, self._sizes[0]), ("scales", scales, self._sizes[1])):
            if t.dtype != torch.uint8 or t.numel() != n:
                raise ValueError("%s must be uint8 with %d elements" % (name, n))
        self._index = -1 if not (codes.is_cuda and scales.is_cuda) else _device(codes, scales)
        self._hold, self._pc, self._ps = (codes, scales), codes.data_ptr(), scales.data_ptr()

    def _shape(self, rows, nblocks, cols, by_block, code):
        self.rows, self.nblocks, self.cols, self.by_block, self.code = rows, nblocks, cols, by_block, code
        self._layers = {}
        self._sizes = _buffer_bytes(MonarchMx4Dims(rows, nblocks, cols, by_block, code))

    @classmethod
    def _new(cls, like, rows, nblocks, cols, by_block, code, stream):
        """Uninitialised, on like's device: both buffers in one piece of memory."""
        q = cls.__new__(cls)
        q._shape(rows, nblocks, cols, by_block, code)
        at = (q._sizes[0] + 511) & ~511
        q._hold = _empty(like, (at + q._sizes[1],), torch.uint8, stream)
        q._pc = q._hold.data_ptr()
        q._ps = q._pc + at
        q._index = like.get_device()
        return q

    def _memory(self):
        return self._hold[0] if isinstance(self._hold, tuple) else self._hold

    @property
    def codes(self):
        return self._hold[0] if isinstance(self._hold, tuple) else self._hold[:self._sizes[0]]

    @property
    def scales(self):
        return self._hold[1] if isinstance(self._hold, tuple) else self._hold[self._hold.numel() - self._sizes[1]:]

    @property
    def dtype(self) -> str:
        return "bf16" if self.code == MONARCH_BF16 else "f32"

    @property
    def device(self):
        return self.codes.device

    @property
    def shape(self):
        """Shape of the plain tensor."""
        return (self.nblocks, self.rows, self.cols) if self.by_block else (self.rows, self.nblocks * self.cols)

    @property
    def nbytes(self) -> int:
        return sum(self._sizes)

    def __repr__(self):
        return "Mx4(shape=%s, nblocks=%d, dtype=%s)" % (tuple(self.shape), self.nblocks, self.dtype)


def _buffer_bytes(d) -> tuple:
    """(codes, scales) bytes; raises MonarchError on sizes that the library does not take."""
    L, p = lib(), _byref(d)
    codes, scales = L.monarch_mx4_code_bytes(p), L.monarch_mx4_scale_bytes(p)
    if codes == 0 and d.rows != 0:
        _check("monarch_mx4_quantise", L.monarch_mx4_quantise(None, p, None, None, None))
    return codes, scales


# The binding's own cost counts where a kernel takes a few microseconds (a decoding step), so the checks
# below use one call per property and no object that is not needed.
def _device(*ts) -> int:
    """Index of the device that holds every tensor; all must be contiguous CUDA tensors."""
    device = None
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i < 0 or not t.is_contiguous():
                raise ValueError("Monarch kernels take contiguous CUDA tensors")
            if device is None:
                device = i
            elif i != device:
                raise ValueError("tensors on cuda:%d and cuda:%d: one call takes one device's" % (device, i))
    return device


def _together(device, *qs):
    """Raises unless every Mx4 lies on `device`."""
    for q in qs:
        if q is not None and q._index != device:
            raise ValueError("an Mx4 on %s and tensors on cuda:%d: one call takes one device's" % (q.device, device))


def _empty(like, shape, dtype, stream):
    """Memory on like's device for work on `stream` (None: that device's current one)."""
    if stream is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _call(name, fn, device, stream, *args):
    """fn, the C entry point `name`, on args and the stream handle, with `device` the current one."""
    s = _raw_stream(device) if stream is None else stream.cuda_stream
    if device == _current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    if rc:
        _check(name, rc)


def _p(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace, need, like, stream):
    """(tensor to keep alive, address, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty(like, (need,), torch.uint8, stream)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _code(t, name) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError("%s is %s: bfloat16 and float32 are taken" % (name, t.dtype))
    return code


def mx4_quantise(X, nblocks: int | None = None, stream=None) -> Mx4:
    """X in MX4.  A 3-D X is a weight (nblocks, out_blk, in_blk); a 2-D X (rows, nblocks * cols) holds
    activations of `nblocks` blocks (default 1).  Scales never span two rows or two blocks."""
    code = _code(X, "X")
    shape = X.shape
    by_block = len(shape) == 3
    if by_block:
        nb, rows, cols = shape
        if nblocks is not None and nblocks != nb:
            raise ValueError("X has %d blocks, nblocks is %d" % (nb, nblocks))
    elif len(shape) == 2:
        nb = 1 if nblocks is None else int(nblocks)
        rows, width = shape
        if nb <= 0 or width % nb:
            raise ValueError("%d columns do not divide into %d blocks" % (width, nb))
        cols = width // nb
    else:
        raise ValueError("X must have 2 or 3 dimensions, got %d" % len(shape))
    device = _device(X)
    q = Mx4._new(X, rows, nb, cols, by_block, code, stream)
    _call("monarch_mx4_quantise", lib().monarch_mx4_quantise, device, stream, X.data_ptr(),
          _byref(MonarchMx4Dims(rows, nb, cols, by_block, code)), q._pc, q._ps)
    return q


def mx4_dequantise(q: Mx4, dtype=None, out=None, stream=None):
    """The values of q in the layout it came from, in `dtype` (default: the type it came in)."""
    code = q.code if dtype is None else dtype_code(dtype)
    dt = _DTYPES[code]
    if out is None:
        out = _empty(q._memory(), q.shape, dt, stream)
    elif tuple(out.shape) != tuple(q.shape) or out.dtype != dt:
        raise ValueError("out must be %s of shape %s" % (dt, tuple(q.shape)))
    device = _device(out)
    _together(device, q)
    _call("monarch_mx4_dequantise", lib().monarch_mx4_dequantise, device, stream, q._pc, q._ps,
          _byref(MonarchMx4Dims(q.rows, q.nblocks, q.cols, q.by_block, code)), out.data_ptr())
    return out


def _weight(W, name="W"):
    if not isinstance(W, Mx4) or not W.by_block:
        raise ValueError("%s must be an Mx4 weight: mx4_quantise of (nblocks, out_blk, in_blk)" % name)


def _activations(X, W):
    if X.by_block or X.nblocks != W.nblocks or X.cols != W.cols:
        raise ValueError("X is %r, W %r: an Mx4 X must hold activations with W's blocks" % (X, W))


def _expect(t, name, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError("%s must be %s of shape %s, is %s of shape %s" % (name, dtype, shape, t.dtype, tuple(t.shape)))


def _remember(W, key, plan):
    if len(W._layers) >= 64:  # a serving loop sees few batch sizes; any number must not pile up
        W._layers.clear()
    W._layers[key] = plan
    return plan


def _layer(W, rows, has_bias, code):
    """(dims by reference, forward workspace bytes, backward workspace bytes) of a layer with weight W."""
    key = (rows, has_bias, code)
    plan = W._layers.get(key)
    if plan is None:
        d, L = _byref(MonarchMx4LinearDims(rows, W.nblocks, W.cols, W.rows, has_bias, code)), lib()
        plan = _remember(W, key, (d, L.monarch_mx4_linear_wfwd_workspace_bytes(d), L.monarch_mx4_linear_bwd_workspace_bytes(d)))
    return plan


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
    n_out = W.nblocks * W.rows
    if isinstance(X, Mx4):
        _activations(X, W)
        code = X.code if dtype is None else dtype_code(dtype)
        rows, dt = X.rows, _DTYPES[code]
        if bias is not None:
            _expect(bias, "bias", (n_out,), dt)
        if Y is None:
            Y = _empty(X._memory(), (rows, n_out), dt, stream)
        else:
            _expect(Y, "Y", (rows, n_out), dt)
        device = _device(Y, bias)
        _together(device, W, X)
        _call("monarch_mx4_linear_fwd", lib().monarch_mx4_linear_fwd, device, stream, X._pc, X._ps, W._pc, W._ps, _p(bias),
              _layer(W, rows, bias is not None, code)[0], Y.data_ptr())
        return Y
    dt = X.dtype
    code = _code(X, "X")
    if dtype is not None and dtype_code(dtype) != code:
        raise ValueError("dtype is X's unless X is an Mx4")
    rows = X.shape[0]
    if X.shape != (rows, W.nblocks * W.cols):
        _expect(X, "X", (rows, W.nblocks * W.cols), dt)
    if bias is not None:
        _expect(bias, "bias", (n_out,), dt)
    if Y is not None:
        _expect(Y, "Y", (rows, n_out), dt)
    device = _device(X, bias, Y, workspace)
    _together(device, W)
    if Y is None:
        Y = _empty(X, (rows, n_out), dt, stream)
    d, need, _ = _layer(W, rows, bias is not None, code)
    workspace, wp, wn = _workspace(workspace, need, X, stream)
    _call("monarch_mx4_linear_wfwd", lib().monarch_mx4_linear_wfwd, device, stream, X.data_ptr(), W._pc, W._ps, _p(bias), d,
          Y.data_ptr(), wp, wn)
    return Y


def mx4_linear_bwd(dY, X, W, bias: bool = False, need_dX: bool = True, dX=None, dW=None, dbias=None, workspace=None,
                   stream=None):
    """(dX, dW, dbias) of mx4_linear_fwd(X, W) for its quantised operands; a training step passes them on
    to the tensors X and W were rounded from.  X = None (a frozen layer) leaves out dW; need_dX = False
    leaves out dX; dbias is None without `bias`."""
    _weight(W)
    code = _code(dY, "dY")
    dt = dY.dtype
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
    _expect(dY, "dY", (rows, n_out), dt)
    _expect(dX, "dX", (rows, n_in), dt)
    _expect(dW, "dW", (W.nblocks, W.rows, W.cols), dt)
    _expect(dbias, "dbias", (n_out,), dt)
    if not need_dX:
        dX = None
    elif dX is None:
        dX = _empty(dY, (rows, n_in), dt, stream)
    if X is not None and dW is None:
        dW = _empty(dY, (W.nblocks, W.rows, W.cols), dt, stream)
    if not bias:
        dbias = None
    elif dbias is None:
        dbias = _empty(dY, (n_out,), dt, stream)
    device = _device(dY, dX, dW, dbias, workspace)
    _together(device, W, X)
    d, _, need = _layer(W, rows, bool(bias), code)
    workspace, wp, wn = _workspace(workspace, need, dY, stream)
    xc, xs = (None, None) if X is None else (X._pc, X._ps)
    _call("monarch_mx4_linear_bwd", lib().monarch_mx4_linear_bwd, device, stream, dY.data_ptr(), xc, xs, W._pc, W._ps, d, _p(dX),
          _p(dW), _p(dbias), wp, wn)
    return dX, dW, dbias


def mx4_fwd(X, R: Mx4, L: Mx4, shape: dict, Y=None, workspace=None, stream=None):
    """Monarch map Y = X M^T with both factors in MX4 (fwd() with the factors' quantised values)."""
    _weight(R, "R")
    _weight(L, "L")
    nb1, in1, out1, nb2, in2, out2 = shape["nb1"], shape["in1"], shape["out1"], shape["nb2"], shape["in2"], shape["out2"]
    for name, q, want in (("R", R, (nb1, out1, in1)), ("L", L, (nb2, out2, in2))):
        if q.shape != want:
            raise ValueError("%s has shape %s, the dims need %s" % (name, q.shape, want))
    code = _code(X, "X")
    dt = X.dtype
    rows = X.shape[0]
    if X.shape != (rows, nb1 * in1):
        _expect(X, "X", (rows, nb1 * in1), dt)
    if Y is not None:
        _expect(Y, "Y", (rows, nb2 * out2), dt)
    device = _device(X, Y, workspace)
    _together(device, R, L)
    if Y is None:
        Y = _empty(X, (rows, nb2 * out2), dt, stream)
    # R's cache: dims of a map with this factor and its workspace bytes, by what else is in the dims
    key = (rows, code, nb2, in2, out2, shape.get("out_transpose", 1))
    plan = R._layers.get(key)
    if plan is None:
        d = _byref(MonarchDims(rows, nb1, in1, out1, nb2, in2, out2, int(key[-1]), code))
        plan = _remember(R, key, (d, lib().monarch_mx4_fwd_workspace_bytes(d)))
    workspace, wp, wn = _workspace(workspace, plan[1], X, stream)
    _call("monarch_mx4_fwd", lib().monarch_mx4_fwd, device, stream, X.data_ptr(), R._pc, R._ps, L._pc, L._ps, plan[0], Y.data_ptr(),
          wp, wn)
    return Y
