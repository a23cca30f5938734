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
import struct

import torch

from .build import native_key
from . import MONARCH_BF16, MONARCH_F32, MonarchMx4Dims, MonarchMx4LinearDims, _check, dtype_code, lib, make_dims

_ENTRY_POINTS = ("monarch_mx4_code_bytes", "monarch_mx4_scale_bytes", "monarch_mx4_quantise", "monarch_mx4_dequantise",
                 "monarch_mx4_linear_wfwd_workspace_bytes", "monarch_mx4_linear_bwd_workspace_bytes", "monarch_mx4_linear_fwd",
                 "monarch_mx4_linear_wfwd", "monarch_mx4_linear_bwd", "monarch_mx4_fwd_workspace_bytes", "monarch_mx4_fwd")


def _load():
    """The native half (csrc/mx4_native.cpp), given libmonarch's entry points in the order it takes them."""
    L = lib()
    again = "; run `python -m block_diagonal_linear_b200.build`"
    try:
        from . import _mx4_native
    except ImportError as e:
        raise RuntimeError("_mx4_native.so is not built, or not for this torch" + again) from e
    if getattr(_mx4_native, "key", None) != native_key(torch):
        raise RuntimeError("_mx4_native.so is built for %r, this is %r%s" % (getattr(_mx4_native, "key", None), native_key(torch), again))
    _mx4_native.init(tuple(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in _ENTRY_POINTS), _check)
    return _mx4_native


_native = _load()
_RAW = struct.Struct("8q")  # addresses of codes and scales, rows, nblocks, cols, by_block, dtype, device (-1: not CUDA)


class Mx4:
    """A quantised tensor: ``nblocks`` matrices of (rows, cols), scales shared along cols.

    ``codes`` and ``scales`` are contiguous uint8 CUDA tensors in the layout of ``include/monarch.h``;
    ``by_block`` says which plain layout it came from: (nblocks, rows, cols), or (rows, nblocks * cols);
    ``dtype`` is that tensor's type ("bf16" / "f32")."""

    # _hold: what keeps the memory alive; _raw: what the native half takes (_RAW), fixed with the memory
    __slots__ = ("rows", "nblocks", "cols", "by_block", "code", "_hold", "_sizes", "_raw")

    def __init__(self, codes, scales, rows: int, nblocks: int, cols: int, by_block: bool, dtype):
        self.rows, self.nblocks, self.cols, self.by_block = int(rows), int(nblocks), int(cols), bool(by_block)
        self.code = dtype_code(dtype)
        self._sizes = _buffer_bytes(MonarchMx4Dims(self.rows, self.nblocks, self.cols, self.by_block, self.code))
        for name, t, n in (("codes", codes, self._sizes[0]), ("scales", scales, self._sizes[1])):
            if t.dtype != torch.uint8 or t.numel() != n:
                raise ValueError("%s must be uint8 with %d elements" % (name, n))
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)
        if codes.device != scales.device:
            raise ValueError("codes on %s and scales on %s: one device holds both" % (codes.device, scales.device))
        self._hold = (codes, scales)
        self._raw = _RAW.pack(codes.data_ptr(), scales.data_ptr(), self.rows, self.nblocks, self.cols, self.by_block, self.code,
                              codes.get_device() if codes.is_cuda else -1)

    def __reduce__(self):  # copies and pickles: _raw belongs to this object's memory alone
        return Mx4, (self.codes, self.scales, self.rows, self.nblocks, self.cols, self.by_block, self.code)

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
    L, p = lib(), ctypes.byref(d)
    codes, scales = L.monarch_mx4_code_bytes(p), L.monarch_mx4_scale_bytes(p)
    if codes == 0 and d.rows != 0:
        _check("monarch_mx4_quantise", L.monarch_mx4_quantise(None, p, None, None, None))
    return codes, scales


def _on(stream, t, f, *args):
    """f(*args) with `stream`, a stream of t's device, as the current one: its work and memory are the stream's."""
    if stream.device != t.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    with torch.cuda.stream(stream):
        return f(*args)


def _code(dtype) -> int:
    """MONARCH_* code of a type."""
    try:
        code = dtype_code(dtype)
    except KeyError:
        code = None
    if code not in (MONARCH_BF16, MONARCH_F32):
        raise ValueError("dtype %s: bf16 and f32 are taken" % (dtype,))
    return code


def mx4_quantise(X, nblocks: int | None = None, stream=None) -> Mx4:
    """X in MX4.  A 3-D X is a weight (nblocks, out_blk, in_blk); a 2-D X (rows, nblocks * cols) holds
    activations of `nblocks` blocks (default 1).  Scales never span two rows or two blocks."""
    if stream is None:
        hold, raw, codes, scales = _native.quantise(X, nblocks)
    else:
        hold, raw, codes, scales = _on(stream, X, _native.quantise, X, nblocks)
    q = Mx4.__new__(Mx4)
    _, _, q.rows, q.nblocks, q.cols, by_block, q.code, _ = _RAW.unpack(raw)
    q.by_block = by_block == 1
    q._hold, q._raw, q._sizes = hold, raw, (codes, scales)
    return q


def mx4_dequantise(q: Mx4, dtype=None, out=None, stream=None):
    """The values of q in the layout it came from, in `dtype` (default: the type it came in)."""
    if not isinstance(q, Mx4):
        raise ValueError("q must be an Mx4")
    args = (q._raw, q.code if dtype is None else _code(dtype), out)
    return _native.dequantise(*args) if stream is None else _on(stream, q, _native.dequantise, *args)


def _weight(W, name="W"):
    if not isinstance(W, Mx4) or not W.by_block:
        raise ValueError("%s must be an Mx4 weight: mx4_quantise of (nblocks, out_blk, in_blk)" % name)


def _activations(X, W):
    if X.by_block or X.nblocks != W.nblocks or X.cols != W.cols:
        raise ValueError("X is %r, W %r: an Mx4 X must hold activations with W's blocks" % (X, W))


def mx4_linear_workspace_bytes(rows: int, nblocks: int, in_blk: int, out_blk: int, dtype="bf16", bias: bool = False,
                               backward: bool = False) -> int:
    """Workspace of mx4_linear_fwd with a plain X, or of mx4_linear_bwd."""
    d = MonarchMx4LinearDims(int(rows), int(nblocks), int(in_blk), int(out_blk), int(bool(bias)), dtype_code(dtype))
    f = lib().monarch_mx4_linear_bwd_workspace_bytes if backward else lib().monarch_mx4_linear_wfwd_workspace_bytes
    return int(f(ctypes.byref(d)))


_PRODUCTS = {"both": 0, "weights": 1, "dX": 2, "dW": 3}


def mx4_linear_path(product: str, rows: int, nblocks: int, in_blk: int, out_blk: int, dtype="bf16") -> int:
    """Kernels of one product of a layer (host-only query; `include/monarch.h` has the numbers): "both" operands in
    MX4 or the "weights" alone (forward), "dX" or "dW"."""
    d = MonarchMx4LinearDims(int(rows), int(nblocks), int(in_blk), int(out_blk), 0, dtype_code(dtype))
    return lib().monarch_mx4_linear_path(ctypes.byref(d), _PRODUCTS[product])


def mx4_fwd_path(shape: dict, rows: int, dtype="bf16") -> int:
    """Kernels of mx4_fwd (host-only query): 0 the few-token ones, else fwd_path() of the forward behind the expanded factors."""
    return lib().monarch_mx4_fwd_path(ctypes.byref(make_dims(shape, rows, dtype)))


def mx4_linear_fwd(X, W: Mx4, bias=None, Y=None, dtype=None, workspace=None, stream=None):
    """Block-diagonal linear layer with W in MX4: Y[r, b*out + o] = sum_i X[r, b*in + i] W[b, o, i] + bias.

    X is a plain tensor (rows, nblocks * in_blk), or an Mx4 of one; then Y has `dtype` (default: the type
    X was quantised from), and no workspace is needed: one that is given is left as it is."""
    _weight(W)
    if isinstance(X, Mx4):
        _activations(X, W)
        f, args = _native.linear_mx4, (X._raw, W._raw, X.code if dtype is None else _code(dtype), bias, Y)
    else:
        if dtype is not None and _code(dtype) != _code(X.dtype):
            raise ValueError("dtype is X's unless X is an Mx4")
        f, args = _native.linear_plain, (X, W._raw, bias, Y, workspace)
    return f(*args) if stream is None else _on(stream, X, f, *args)


def mx4_linear_bwd(dY, X, W, bias: bool = False, need_dX: bool = True, dX=None, dW=None, dbias=None, workspace=None,
                   stream=None):
    """(dX, dW, dbias) of mx4_linear_fwd(X, W) for its quantised operands; a training step passes them on
    to the tensors X and W were rounded from.  X = None (a frozen layer) leaves out dW; need_dX = False
    leaves out dX; dbias is None without `bias`.  A buffer for a gradient that is not asked for is refused."""
    _weight(W)
    if X is not None:
        if not isinstance(X, Mx4):
            raise ValueError("X must be the forward's Mx4 X, or None")
        _activations(X, W)
    args = (dY, None if X is None else X._raw, W._raw, need_dX, bias, dX, dW, dbias, workspace)
    return _native.linear_bwd(*args) if stream is None else _on(stream, dY, _native.linear_bwd, *args)


def mx4_fwd(X, R: Mx4, L: Mx4, shape: dict, Y=None, workspace=None, stream=None):
    """Monarch map Y = X M^T with both factors in MX4 (fwd() with the factors' quantised values)."""
    _weight(R, "R")
    _weight(L, "L")
    dims = (shape["nb1"], shape["in1"], shape["out1"], shape["nb2"], shape["in2"], shape["out2"], shape.get("out_transpose", 1))
    args = (X, R._raw, L._raw, dims, Y, workspace)
    return _native.monarch(*args) if stream is None else _on(stream, X, _native.monarch, *args)
