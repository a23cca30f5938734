"""MX4 operators without a GPU: the oracle's pins, the buffer sizes, and every refusal of the C entry
points and the binding (fake device pointers: each call must fail before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import block_diagonal_linear_b200 as bdl
import oracle

CODES = bdl.CODES


# ---------------------------------------------------------------- oracle pins
def test_oracle_rounds_hand_values():
    # the largest magnitude 6 gives scale 2^0, so the values are rounded on the grid itself
    x = np.zeros(32)
    x[:16] = [6, 5, 4.99, 5.01, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -0.25, -0.75, -5, 3.4, -2.6]
    want = [6, 4, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, 0, -1, -4, 3, -3]
    assert oracle.mx4_round(x)[:16].tolist() == want
    assert oracle.mx4_encode(x)[1].tolist() == [127]


def test_oracle_scale_rule():
    for top, byte in ((1.0, 125), (7.9, 127), (8.0, 128), (0.0, 0), (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1),
                      (2.0 ** -149, 0), (3.3e38, 252)):
        x = np.zeros(32)
        x[3] = -top
        assert oracle.mx4_encode(x)[1].tolist() == [byte], top
    assert oracle.mx4_round(np.array([7.9]))[0] == 6.0     # cut at 6 times the scale
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones(40)
        x[5] = bad
        v = oracle.mx4_round(x)
        assert np.isnan(v[:32]).all() and (v[32:] == 1).all()


def test_oracle_rounding_is_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 1)))
    codes, scales = oracle.mx4_encode(x)
    v = oracle.mx4_decode(codes, scales, 96)
    s = np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=1)
    a = np.minimum(np.abs(x) / s, 6)
    best = np.abs(a[..., None] - oracle.MX4_GRID).min(-1)
    assert np.allclose(np.abs(a - np.abs(v) / s), best, atol=0)
    assert (np.abs(x).reshape(64, 3, 32).max(-1) / s[:, ::32] < 8).all()


def test_oracle_linear_backward_against_differences():
    rng = np.random.default_rng(1)
    X, W, dY = rng.standard_normal((5, 6)), rng.standard_normal((2, 4, 3)), rng.standard_normal((5, 8))
    dX, dW, db = oracle.mx4_linear_backward(dY, X, W)
    f = lambda X, W, b: float((oracle.mx4_linear_forward(X, W, b) * dY).sum())  # noqa: E731
    b, h = np.zeros(8), 0.5  # linear in each operand: differences are exact but for rounding
    for arr, grad in ((X, dX), (W, dW), (b, db)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = f(X, W, b)
            arr[i] = keep - h
            down = f(X, W, b)
            arr[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-12


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("rows,nb,cols,codes,scales", [
    (1, 1, 1, 16, 512), (1, 1, 32, 16, 512), (128, 2, 128, 2 * 128 * 64, 2 * 512),
    (129, 3, 129, 3 * 129 * 80, 3 * 2 * 2 * 512), (0, 4, 64, 0, 0)])
def test_buffer_sizes(rows, nb, cols, codes, scales):
    d = bdl.MonarchMx4Dims(rows, nb, cols, 1, bdl.MONARCH_BF16)
    assert bdl.lib().monarch_mx4_code_bytes(ctypes.byref(d)) == codes
    assert bdl.lib().monarch_mx4_scale_bytes(ctypes.byref(d)) == scales
    p, s = oracle.mx4_buffers(np.ones((nb, rows, cols)))
    assert (p.size, s.size) == (codes, scales)


# ---------------------------------------------------------------- C refusals
P = ctypes.c_void_p


def at(k):
    return P((k + 1) << 40)


def test_quantise_refusals():
    L = bdl.lib()
    D = bdl.MonarchMx4Dims
    good = D(4, 2, 64, 0, bdl.MONARCH_F32)

    def q(d, X=at(0), c=at(1), s=at(2)):
        rcs = (L.monarch_mx4_quantise(X, ctypes.byref(d) if d is not None else None, c, s, None),
               L.monarch_mx4_dequantise(c, s, ctypes.byref(d) if d is not None else None, X, None))
        assert rcs[0] == rcs[1]
        return rcs[0]

    assert q(None) == CODES["MONARCH_ERR_NULL"]
    assert q(D(4, 2, 64, 0, 2)) == CODES["MONARCH_ERR_DTYPE"]
    for bad in (D(-1, 2, 64, 0, 0), D(4, 0, 64, 0, 0), D(4, 2, 0, 0, 0)):
        assert q(bad) == CODES["MONARCH_ERR_DIMS"]
        assert L.monarch_mx4_code_bytes(ctypes.byref(bad)) == 0
    for big in (D(2 ** 31 - 255, 1, 32, 0, 0), D(1, 65536, 32, 0, 0), D(1, 1, 2 ** 20 + 1, 0, 0), D(1, 5, 2 ** 20, 0, 0)):
        assert q(big) == CODES["MONARCH_ERR_UNSUPPORTED"]
    assert q(good, X=None) == q(good, c=None) == q(good, s=None) == CODES["MONARCH_ERR_NULL"]
    assert q(good, X=P(4104)) == q(good, c=P(4104)) == q(good, s=P(4104)) == CODES["MONARCH_ERR_ALIGN"]
    assert q(good, X=at(0), c=P((1 << 40) + 16)) == CODES["MONARCH_ERR_ALIAS"]
    assert L.monarch_mx4_quantise(at(0), ctypes.byref(good), at(1), at(1), None) == CODES["MONARCH_ERR_ALIAS"]
    assert q(D(0, 2, 64, 0, 0), X=None, c=None, s=None) == 0


def test_linear_refusals():
    L = bdl.lib()
    D = bdl.MonarchMx4LinearDims

    def f(d, xc=at(0), xs=at(1), wc=at(2), ws=at(3), b=at(4), Y=at(5)):
        return L.monarch_mx4_linear_fwd(xc, xs, wc, ws, b, ctypes.byref(d) if d is not None else None, Y, None)

    def w(d, X=at(0), wc=at(2), ws=at(3), b=at(4), Y=at(5), work=at(6), n=None):
        n = L.monarch_mx4_linear_wfwd_workspace_bytes(ctypes.byref(d)) if n is None and d is not None else n or 0
        return L.monarch_mx4_linear_wfwd(X, wc, ws, b, ctypes.byref(d) if d is not None else None, Y, work, n, None)

    good = D(40, 2, 64, 96, 1, bdl.MONARCH_BF16)
    for g in (f, w):
        assert g(None) == CODES["MONARCH_ERR_NULL"]
        assert g(D(40, 2, 64, 96, 0, 5)) == CODES["MONARCH_ERR_DTYPE"]
        for bad in (D(-1, 2, 64, 96, 0, 0), D(4, 0, 64, 96, 0, 0), D(4, 2, 0, 96, 0, 0), D(4, 2, 64, -3, 0, 0)):
            assert g(bad) == CODES["MONARCH_ERR_DIMS"]
            assert L.monarch_mx4_linear_wfwd_workspace_bytes(ctypes.byref(bad)) == 0
            assert L.monarch_mx4_linear_bwd_workspace_bytes(ctypes.byref(bad)) == 0
        assert g(D(4, 2, 64, 2 ** 20 + 1, 0, 0)) == CODES["MONARCH_ERR_UNSUPPORTED"]
        for name in ("wc", "ws", "b", "Y"):
            assert g(good, **{name: None}) == CODES["MONARCH_ERR_NULL"]
            assert g(good, **{name: P(4100)}) == CODES["MONARCH_ERR_ALIGN"]
        assert g(good, Y=P((3 << 40) + 32)) == CODES["MONARCH_ERR_ALIAS"]      # W's codes
        assert g(good, Y=P((5 << 40) - 16)) == CODES["MONARCH_ERR_ALIAS"]      # into the bias
        assert g(D(0, 2, 64, 96, 1, 1), wc=None, ws=None, b=None, Y=None) == 0
    long = D(700, 2, 640, 960, 1, bdl.MONARCH_BF16)   # many rows of a large weight: its values are expanded in a workspace
    need = L.monarch_mx4_linear_wfwd_workspace_bytes(ctypes.byref(long))
    assert need > 0 and L.monarch_mx4_linear_wfwd_workspace_bytes(ctypes.byref(good)) == 0
    assert w(long, work=None) == w(long, n=need - 1) == CODES["MONARCH_ERR_WORKSPACE"]
    assert w(long, work=P((7 << 40) + 16)) == CODES["MONARCH_ERR_ALIGN"]
    assert w(long, work=at(0)) == w(long, work=at(2)) == w(long, work=at(5)) == CODES["MONARCH_ERR_ALIAS"]
    assert f(good, xc=None) == f(good, xs=None) == w(good, X=None) == CODES["MONARCH_ERR_NULL"]
    assert f(good, xc=P(8)) == f(good, xs=P(8)) == w(good, X=P(8)) == CODES["MONARCH_ERR_ALIGN"]


def test_linear_backward_refusals():
    L = bdl.lib()
    D = bdl.MonarchMx4LinearDims
    good = D(40, 2, 64, 96, 1, bdl.MONARCH_BF16)
    need = L.monarch_mx4_linear_bwd_workspace_bytes(ctypes.byref(good))
    assert need > 0

    def g(d=good, dY=at(0), xc=at(1), xs=at(2), wc=at(3), ws=at(4), dX=at(5), dW=at(6), db=at(7), work=at(8), n=need):
        return L.monarch_mx4_linear_bwd(dY, xc, xs, wc, ws, ctypes.byref(d) if d is not None else None, dX, dW, db, work, n, None)

    assert g(None) == CODES["MONARCH_ERR_NULL"]
    assert g(D(40, 2, 64, 96, 1, 3)) == CODES["MONARCH_ERR_DTYPE"]
    assert g(D(40, 2, 64, 0, 1, 1)) == CODES["MONARCH_ERR_DIMS"]
    for name in ("dY", "xc", "xs", "wc", "ws", "db"):
        assert g(**{name: None}) == CODES["MONARCH_ERR_NULL"], name
    for name in ("dY", "xc", "xs", "wc", "ws", "dX", "dW", "db"):
        assert g(**{name: P(4104)}) == CODES["MONARCH_ERR_ALIGN"], name
    assert g(work=None) == g(n=need - 1) == CODES["MONARCH_ERR_WORKSPACE"]
    assert g(work=P((9 << 40) + 16)) == CODES["MONARCH_ERR_ALIGN"]
    for name in ("dX", "dW", "db", "work"):
        assert g(**{name: at(0)}) == CODES["MONARCH_ERR_ALIAS"], name     # dY
        assert g(**{name: at(3)}) == CODES["MONARCH_ERR_ALIAS"], name     # W's codes
    assert g(dX=at(6)) == CODES["MONARCH_ERR_ALIAS"]


def test_monarch_refusals():
    L = bdl.lib()
    shape = dict(nb1=4, in1=64, out1=32, nb2=4, in2=32, out2=96, out_transpose=0)
    good = bdl.make_dims(shape, 7, "bf16")
    need = L.monarch_mx4_fwd_workspace_bytes(ctypes.byref(good))
    assert need > 0

    def g(d=good, X=at(0), rc=at(1), rs=at(2), lc=at(3), ls=at(4), Y=at(5), work=at(6), n=need):
        return L.monarch_mx4_fwd(X, rc, rs, lc, ls, ctypes.byref(d) if d is not None else None, Y, work, n, None)

    assert g(None) == CODES["MONARCH_ERR_NULL"]
    assert g(bdl.make_dims(dict(shape, out1=31), 7, "bf16")) == CODES["MONARCH_ERR_DIMS"]
    assert g(bdl.make_dims(shape, 7, 9)) == CODES["MONARCH_ERR_DTYPE"]
    for name in ("X", "rc", "rs", "lc", "ls", "Y"):
        assert g(**{name: None}) == CODES["MONARCH_ERR_NULL"], name
        assert g(**{name: P(4104)}) == CODES["MONARCH_ERR_ALIGN"], name
    assert g(work=None) == g(n=need - 1) == CODES["MONARCH_ERR_WORKSPACE"]
    assert g(work=P((7 << 40) + 64)) == CODES["MONARCH_ERR_ALIGN"]
    for name in ("Y", "work"):
        for k in (0, 1, 3):
            assert g(**{name: at(k)}) == CODES["MONARCH_ERR_ALIAS"], (name, k)
    assert g(bdl.make_dims(shape, 0, "bf16"), X=None, Y=None) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_monarch_rows_beyond_one_launch_keep_their_kernels(dtype):
    """Factors that the plain forward has no tensor-core kernel for, here none at all: the few-token kernels take any number
    of rows, so many at a time, in one and the same workspace."""
    L = bdl.lib()
    shape = dict(nb1=1, in1=8, out1=60000, nb2=1, in2=60000, out2=8, out_transpose=0)
    assert bdl.fwd_path(shape, dtype) == 0
    need = [L.monarch_mx4_fwd_workspace_bytes(ctypes.byref(bdl.make_dims(shape, r, dtype))) for r in (65536, 65537, 524280, 524281, 1 << 24)]
    assert need == [65536 * 60000 * 4] * 5
    assert L.monarch_mx4_fwd_workspace_bytes(ctypes.byref(bdl.make_dims(shape, 100, dtype))) == 100 * 60000 * 4


def test_path_queries():
    from test_gpu_mx4 import PATHS
    reached = {}
    for product, rows, nb, inn, out, dtype, path in PATHS:
        assert bdl.mx4_linear_path(product, rows, nb, inn, out, dtype) == path
        reached.setdefault(product, set()).add(path)
    # every kernel but the direct few-token one, which the small layers take
    assert reached == {"both": {2, 3, 4, 5, 6, 7}, "weights": {1, 8, 9, 24, 25}, "dX": {9, 24, 25}, "dW": {9, 24, 25}}
    assert bdl.mx4_linear_path("both", 1, 1, 64, 64) == bdl.mx4_linear_path("weights", 1, 1, 64, 64) == 0
    assert bdl.mx4_linear_path("dX", 100, 1, 64, 64) == bdl.mx4_linear_path("dW", 100, 1, 64, 64) == 8
    L = bdl.lib()
    good, bad = bdl.MonarchMx4LinearDims(4, 1, 64, 64, 0, 0), bdl.MonarchMx4LinearDims(4, 0, 64, 64, 0, 0)
    assert L.monarch_mx4_linear_path(None, 0) == L.monarch_mx4_linear_path(ctypes.byref(bad), 0) == -1
    assert L.monarch_mx4_linear_path(ctypes.byref(good), 4) == L.monarch_mx4_linear_path(ctypes.byref(good), -1) == -1
    shape = dict(nb1=32, in1=32, out1=32, nb2=32, in2=32, out2=32, out_transpose=1)
    assert [bdl.mx4_fwd_path(shape, r, "bf16") for r in (1, 64, 5000)] == [0, 0, 2] and bdl.mx4_fwd_path(shape, 5000, "f32") == 0
    assert bdl.mx4_fwd_path(dict(shape, in2=31), 5, "bf16") == L.monarch_mx4_fwd_path(None) == -1


# ---------------------------------------------------------------- binding refusals (CPU tensors)
def fake(rows, nb, cols, by_block, dtype="bf16"):
    d = bdl.MonarchMx4Dims(rows, nb, cols, int(by_block), bdl.dtype_code(dtype))
    L = bdl.lib()
    return bdl.Mx4(torch.zeros(L.monarch_mx4_code_bytes(ctypes.byref(d)), dtype=torch.uint8),
                   torch.zeros(L.monarch_mx4_scale_bytes(ctypes.byref(d)), dtype=torch.uint8), rows, nb, cols, by_block, dtype)


def test_binding_refuses_wrong_tensors():
    W = fake(96, 2, 64, True)
    assert W.shape == (2, 96, 64) and W.nbytes == 2 * 96 * 32 + 2 * 512
    with pytest.raises(ValueError):
        bdl.mx4_quantise(torch.zeros(4, 4))                          # not on a GPU
    with pytest.raises(ValueError):
        bdl.mx4_quantise(torch.zeros(4, 6), nblocks=4)
    with pytest.raises(ValueError):
        bdl.mx4_quantise(torch.zeros(4))
    with pytest.raises(ValueError):
        bdl.mx4_quantise(torch.zeros(3, 4, 4), nblocks=2)
    with pytest.raises(ValueError):
        bdl.mx4_quantise(torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(ValueError):
        bdl.Mx4(W.codes[1:], W.scales, 96, 2, 64, True, "bf16")
    X = torch.zeros(5, 128, dtype=torch.bfloat16)
    for bad in (dict(X=X[:, :127]), dict(X=X, W=X), dict(X=fake(5, 1, 128, False)), dict(X=fake(5, 2, 64, True)),
                dict(X=X, bias=torch.zeros(192)), dict(X=X, bias=torch.zeros(191, dtype=torch.bfloat16)),
                dict(X=X, Y=torch.zeros(5, 191, dtype=torch.bfloat16)), dict(X=X, dtype="f32")):
        with pytest.raises(ValueError):
            bdl.mx4_linear_fwd(**{"W": W, **bad})
    dY = torch.zeros(5, 192, dtype=torch.bfloat16)
    Xq = fake(5, 2, 64, False)
    for bad in (dict(X=X), dict(X=fake(6, 2, 64, False)), dict(dY=dY[:, 1:]), dict(W=Xq), dict(dX=dY), dict(dW=dY),
                dict(X=None, dW=torch.zeros(2, 96, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            bdl.mx4_linear_bwd(**{"dY": dY, "X": Xq, "W": W, **bad})
    shape = dict(nb1=2, in1=64, out1=96, nb2=2, in2=96, out2=32, out_transpose=0)
    R, Lf = fake(96, 2, 64, True), fake(32, 2, 96, True)
    for bad in (dict(R=Lf), dict(L=R), dict(X=X[:, 1:]), dict(R=X), dict(Y=torch.zeros(5, 64))):
        with pytest.raises(ValueError):
            bdl.mx4_fwd(**{"X": X, "R": R, "L": Lf, "shape": shape, **bad})


def test_binding_refuses_streams_and_memory_of_other_devices():
    """Host checks ahead of any allocation: stand-ins for a stream and for another device's tensors."""
    class Stream:
        device = torch.device("cuda", 3)
    W, X = fake(96, 2, 64, True), torch.zeros(5, 128, dtype=torch.bfloat16)
    Xq = fake(5, 2, 64, False)
    shape = dict(nb1=2, in1=64, out1=96, nb2=2, in2=96, out2=32, out_transpose=0)
    for call in (lambda: bdl.mx4_quantise(X, nblocks=2, stream=Stream()), lambda: bdl.mx4_dequantise(Xq, stream=Stream()),
                 lambda: bdl.mx4_linear_fwd(X, W, stream=Stream()), lambda: bdl.mx4_linear_fwd(Xq, W, stream=Stream()),
                 lambda: bdl.mx4_linear_bwd(X, Xq, W, stream=Stream()),
                 lambda: bdl.mx4_fwd(X, W, fake(32, 2, 96, True), shape, stream=Stream())):
        with pytest.raises(ValueError, match="the stream is on cuda:3"):
            call()
    for call in (lambda: bdl.mx4_dequantise(Xq), lambda: bdl.mx4_linear_fwd(Xq, W)):  # memory of the host
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call()
    n = W.codes.numel()
    with pytest.raises(ValueError, match="contiguous"):
        bdl.Mx4(torch.zeros(2 * n, dtype=torch.uint8)[::2], W.scales, 96, 2, 64, True, "bf16")
    with pytest.raises(ValueError, match="one device"):
        bdl.Mx4(torch.zeros(n, dtype=torch.uint8, device="meta"), W.scales, 96, 2, 64, True, "bf16")
    for bad in (0, -1, 3):
        with pytest.raises(ValueError, match="do not divide"):
            bdl.mx4_quantise(X, nblocks=bad)
    for bad in (torch.float16, "fp8", 7):
        with pytest.raises(ValueError, match="bf16 and f32"):
            bdl.mx4_dequantise(Xq, bad)
        with pytest.raises(ValueError, match="bf16 and f32"):
            bdl.mx4_linear_fwd(Xq, W, dtype=bad)
    with pytest.raises(ValueError, match="neither bfloat16 nor float32"):
        bdl.mx4_quantise(X.half(), nblocks=2)
    for bad in (None, 3.0, [1]):
        with pytest.raises(ValueError):
            bdl.mx4_quantise(bad)
        with pytest.raises(ValueError):
            bdl.mx4_linear_fwd(bad, W)
        with pytest.raises(ValueError):
            bdl.mx4_linear_bwd(bad, Xq, W)
        with pytest.raises(ValueError):
            bdl.mx4_dequantise(bad)


def test_backward_refuses_buffers_that_it_would_not_fill():
    W, Xq = fake(96, 2, 64, True), fake(5, 2, 64, False)
    dY, dX = torch.zeros(5, 192, dtype=torch.bfloat16), torch.zeros(5, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="need_dX is false"):
        bdl.mx4_linear_bwd(dY, Xq, W, need_dX=False, dX=dX)
    with pytest.raises(ValueError, match="bias is false"):
        bdl.mx4_linear_bwd(dY, Xq, W, dbias=torch.zeros(192, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dW needs X"):
        bdl.mx4_linear_bwd(dY, None, W, dW=torch.zeros(2, 96, 64, dtype=torch.bfloat16))
    for name in ("need_dX", "bias"):
        with pytest.raises(ValueError, match=name + " must be true or false"):
            bdl.mx4_linear_bwd(dY, Xq, W, **{name: torch.zeros(2)})


def test_copies_have_memory_of_their_own():
    import copy
    import pickle
    q = fake(96, 2, 64, True)
    q.codes[3] = 7
    for c in (copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
        assert c.codes.data_ptr() != q.codes.data_ptr() and torch.equal(c.codes, q.codes) and torch.equal(c.scales, q.scales)
        assert c._raw != q._raw and c._raw[16:] == q._raw[16:]
        assert int.from_bytes(c._raw[:8], "little") == c.codes.data_ptr()
        assert int.from_bytes(c._raw[8:16], "little") == c.scales.data_ptr()
        assert (c.shape, c.dtype, c.nbytes) == (q.shape, q.dtype, q.nbytes)
    assert copy.copy(q)._raw == q._raw
