"""MX4 operators on the GPU against the float64 oracle.

Rounding to MX4 is exact arithmetic (a power-of-two scale, one rounding), so codes, scales and values
are compared for equality.  Products are compared element by element with
    |Y - ref| <= half * |ref| + terms * 2^-23 * sum |factors|  (+ the smallest normal number),
where half is the result type's half step (2^-8 bf16, 2^-24 fp32) and `terms` the length of the sum:
each of its fp32 additions is off by at most 2^-23 of a partial sum (2^-24 if it rounds, twice that if
it cuts off), and no partial sum exceeds the sum of the magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import block_diagonal_linear_b200 as bdl
import oracle

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dtype):
    """A float64 array on the GPU in `dtype`, and the values it has there."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(TORCH[dtype]).cuda()
    return t, f64(t)


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, mags, terms, dtype, what, extra=0.0):
    g = f64(got)
    assert g.shape == ref.shape
    tol = HALF[dtype] * np.abs(ref) + (terms * 2.0 ** -23) * mags + 2.0 ** -126 + extra
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, first %s: %r, want %r +- %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], ref[bad][0], tol[bad][0])


def hard_values(rng, shape):
    """Values over the whole range of exponents: ties, cut values, zeros, subnormals."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-30, 30, shape[:-1] + (1,)))
    kind = rng.integers(0, 8, shape)
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, -0.0, x)
    steps = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.75], shape) * rng.choice([-1, 1], shape)
    return np.where(kind >= 5, steps * np.exp2(rng.integers(-3, 3, shape)), x)


SIZES = [(1, 1, 1), (1, 1, 32), (1, 7, 33), (2, 3, 31), (3, 128, 128), (2, 129, 100), (1, 300, 1000), (5, 64, 4),
         (1, 1, 4096), (4, 130, 264), (7, 65, 257)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("by_block", [True, False])
@pytest.mark.parametrize("nb,rows,cols", SIZES)
def test_quantise_equals_oracle(nb, rows, cols, by_block, dtype):
    rng = np.random.default_rng(rows * 1000 + cols)
    X = hard_values(rng, (nb, rows, cols))
    t, v = dev(X if by_block else X.transpose(1, 0, 2).reshape(rows, nb * cols), dtype)
    b = v if by_block else v.reshape(rows, nb, cols).transpose(1, 0, 2)
    q = bdl.mx4_quantise(t) if by_block else bdl.mx4_quantise(t, nblocks=nb)
    codes, scales = oracle.mx4_buffers(b)
    assert np.array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
    want = oracle.mx4_round(b)
    if not by_block:
        want = want.transpose(1, 0, 2).reshape(rows, nb * cols)
    for out in ("bf16", "f32"):
        assert np.array_equal(f64(bdl.mx4_dequantise(q, out)), want)
    assert bdl.mx4_dequantise(q).dtype == t.dtype


def test_quantise_special_values():
    """Subnormals, the largest finite values, and blocks with an infinity or a NaN."""
    X = np.zeros((1, 8, 96))
    X[0, 0, :4] = [2.0 ** -149, 2.0 ** -140, -2.0 ** -133, 2.0 ** -130]
    X[0, 1, :3] = [2.0 ** -126, 2.0 ** -127, -3 * 2.0 ** -128]
    X[0, 2, :3] = [3.3e38, -3e38, 1e38]
    X[0, 3, :] = 1.0
    X[0, 3, 40] = np.inf
    X[0, 4, 7] = np.nan
    X[0, 5, 95] = -np.inf
    X[0, 6, 3] = 1e30
    X[0, 6, 4] = 1e-30
    for dtype in ("bf16", "f32"):
        t, v = dev(X, dtype)
        q = bdl.mx4_quantise(t)
        codes, scales = oracle.mx4_buffers(v)
        assert np.array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)
        assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
        assert np.array_equal(f64(bdl.mx4_dequantise(q)), oracle.mx4_round(v), equal_nan=True)


def test_quantised_again_is_the_same():
    t, _ = dev(np.random.default_rng(3).standard_normal((40, 300)), "bf16")
    once = bdl.mx4_dequantise(bdl.mx4_quantise(t, nblocks=3))
    # a second rounding may only raise the scale's resolution, never move a value
    assert torch.equal(once, bdl.mx4_dequantise(bdl.mx4_quantise(once, nblocks=3)))


# ---------------------------------------------------------------- products
def layer(rows, nb, inn, out, bias, dtype, seed=0):
    """Device tensors of a layer and the float64 values that its quantised operands have."""
    rng = np.random.default_rng(seed + 7 * rows + inn + out)
    X = rng.standard_normal((rows, nb * inn)) * np.where(rng.random(nb * inn) < 0.05, 12.0, 1.0)
    W = rng.uniform(-1, 1, (nb, out, inn)) / np.sqrt(inn)
    t = {}
    t["X"], x = dev(X, dtype)
    t["W"], w = dev(W, dtype)
    t["dY"], dy = dev(rng.standard_normal((rows, nb * out)), dtype)
    t["b"], b = dev(rng.standard_normal(nb * out), dtype)
    if not bias:
        t["b"], b = None, None
    xr = oracle.mx4_round(x.reshape(rows, nb, inn)).reshape(rows, nb * inn)
    return t, dict(x=x, xr=xr, w=oracle.mx4_round(w), dy=dy, b=b)


def check_forward(Y, x, v, inn, dtype, what):
    ref = oracle.mx4_linear_forward(x, v["w"], v["b"])
    mags = oracle.mx4_linear_forward(np.abs(x), np.abs(v["w"]), None if v["b"] is None else np.abs(v["b"]))
    close(Y, ref, mags, inn + 2, dtype, what)


LAYERS = [  # (rows, nblocks, in, out, bias)
    (1, 1, 1, 1, True), (1, 1, 32, 8, False), (1, 4, 256, 1024, True), (2, 3, 200, 500, True), (5, 1, 33, 130, False),
    (8, 2, 64, 64, False), (9, 1, 1000, 72, True), (33, 4, 250, 100, True), (64, 2, 512, 256, False),
    (65, 1, 640, 96, True), (127, 2, 96, 200, True), (128, 1, 128, 128, False), (129, 2, 160, 192, True),
    (200, 16, 48, 48, False), (300, 1, 2048, 384, True), (257, 3, 64, 320, True), (513, 1, 320, 129, False),
    (700, 2, 256, 512, True), (1024, 1, 512, 1024, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb,inn,out,bias", LAYERS)
def test_linear_forward_both_quantised(rows, nb, inn, out, bias, dtype):
    t, v = layer(rows, nb, inn, out, bias, dtype)
    Wq, Xq = bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(t["X"], nblocks=nb)
    Y = bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"])
    assert bdl.last_device_status() == 0
    check_forward(Y, v["xr"], v, inn, dtype, "Y")
    assert torch.equal(Y, bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"]))


# one to four stages of K over many row tiles (a tile of W is kept), last tiles of rows and columns not full
@pytest.mark.parametrize("rows,nb,inn,out,bias,dtype", [
    (19001, 1, 90, 256, True, "bf16"), (19001, 1, 90, 256, True, "f32"), (6000, 2, 288, 1000, False, "f32"),
    (1300, 1, 700, 3840, True, "bf16"), (2333, 1, 1000, 2000, True, "bf16"), (19011, 1, 1024, 240, False, "bf16")])
def test_linear_forward_of_many_rows(rows, nb, inn, out, bias, dtype):
    test_linear_forward_both_quantised(rows, nb, inn, out, bias, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb,inn,out,bias", LAYERS)
def test_linear_forward_weights_only(rows, nb, inn, out, bias, dtype):
    t, v = layer(rows, nb, inn, out, bias, dtype, seed=1)
    Wq = bdl.mx4_quantise(t["W"])
    Y = bdl.mx4_linear_fwd(t["X"], Wq, bias=t["b"])
    assert bdl.last_device_status() == 0
    check_forward(Y, v["x"], v, inn, dtype, "Y")
    assert torch.equal(Y, bdl.mx4_linear_fwd(t["X"], Wq, bias=t["b"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb,inn,out,bias", LAYERS)
def test_linear_backward(rows, nb, inn, out, bias, dtype):
    t, v = layer(rows, nb, inn, out, bias, dtype, seed=2)
    Wq, Xq = bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(t["X"], nblocks=nb)
    got = bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=bias)
    assert bdl.last_device_status() == 0
    ref = oracle.mx4_linear_backward(v["dy"], v["xr"], v["w"])
    mags = oracle.mx4_linear_backward(np.abs(v["dy"]), np.abs(v["xr"]), np.abs(v["w"]))
    for g, r, m, terms, what in zip(got, ref, mags, (out, rows, rows), ("dX", "dW", "dbias")):
        if what == "dbias" and not bias:
            assert g is None
            continue
        close(g, r, m, terms + 2, dtype, what)
    again = bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=bias)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
    # the parts alone: a frozen layer's dX, and dW without dX
    dX, dW, _ = bdl.mx4_linear_bwd(t["dY"], None, Wq)
    assert dW is None and torch.equal(dX, got[0])
    dX, dW, _ = bdl.mx4_linear_bwd(t["dY"], Xq, Wq, need_dX=False)
    assert dX is None and torch.equal(dW, got[1])


# long prompts: the weight expanded, X in place or staged, K split or not
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb,inn,out,bias", [
    (900, 2, 333, 500, True), (1500, 3, 200, 129, False), (2000, 1, 100, 700, True), (1100, 1, 1000, 72, True), (600, 2, 250, 1000, True),
    (70, 3, 1100, 900, False), (400, 1, 3000, 100, True)])
def test_linear_forward_of_a_prompt(rows, nb, inn, out, bias, dtype):
    test_linear_forward_weights_only(rows, nb, inn, out, bias, dtype)


# few tokens, small weights: fewer tiles than warps, blocks in their place, shares of one to four scale tiles
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb,inn,out,bias", [
    (12, 20, 70, 5, True), (30, 9, 300, 24, True), (20, 1, 1500, 64, False), (31, 1, 2048, 40, True), (9, 65, 128, 17, True),
    (32, 3, 33, 128, True), (17, 2, 1030, 16, False), (25, 7, 513, 100, True), (8, 1, 4096, 3, True)])
def test_linear_forward_of_few_tokens(rows, nb, inn, out, bias, dtype):
    test_linear_forward_weights_only(rows, nb, inn, out, bias, dtype)
    test_linear_forward_both_quantised(rows, nb, inn, out, bias, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 9, 40])
def test_few_quantised_tokens_agree_with_many(rows, dtype):
    """The first rows of a long batch and those rows alone: other kernels, sums of the same exact products."""
    t, v = layer(600, 2, 1056, 200, True, dtype, seed=6)
    Wq = bdl.mx4_quantise(t["W"])
    long = bdl.mx4_linear_fwd(bdl.mx4_quantise(t["X"], nblocks=2), Wq, bias=t["b"])
    alone = bdl.mx4_linear_fwd(bdl.mx4_quantise(t["X"][:rows], nblocks=2), Wq, bias=t["b"])
    short = {k: (x[:rows] if k in ("x", "xr", "dy") else x) for k, x in v.items()}
    check_forward(alone, short["xr"], short, 1056, dtype, "Y of a few rows")
    check_forward(long[:rows], short["xr"], short, 1056, dtype, "first rows of a long batch")


# dbias beside dX's product: aligned rows, odd ones, fp32 parts; in a stream of calls that share a workspace, and replayed
@pytest.mark.parametrize("rows,nb,inn,out,dtype", [
    (1300, 1, 512, 1000, "bf16"), (900, 3, 384, 333, "bf16"), (1025, 1, 1024, 1100, "bf16"), (600, 2, 256, 501, "f32")])
def test_linear_backward_of_a_long_batch(rows, nb, inn, out, dtype):
    test_linear_backward(rows, nb, inn, out, True, dtype)
    t, _ = layer(rows, nb, inn, out, True, dtype, seed=3)
    Wq, Xq = bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(t["X"], nblocks=nb)
    steps = [t["dY"] * k for k in (1, -2, 0.5, 4)]  # exact multiples: so are the results
    first = bdl.mx4_linear_bwd(steps[0], Xq, Wq, bias=True)
    ws = torch.empty(bdl.mx4_linear_workspace_bytes(rows, nb, inn, out, dtype, bias=True, backward=True), dtype=torch.uint8, device="cuda")
    given = torch.empty_like(steps[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = bdl.mx4_linear_bwd(given, Xq, Wq, bias=True, workspace=ws)
    for _ in range(3):
        outs = [bdl.mx4_linear_bwd(d, Xq, Wq, bias=True, workspace=ws) for d in steps]
        for d, o, k in zip(steps, outs, (1, -2, 0.5, 4)):
            given.copy_(d)
            graph.replay()
            assert all(torch.equal(a, b * k) and torch.equal(c, a) for a, b, c in zip(o, first, kept))
    assert bdl.last_device_status() == 0


def test_backward_against_differences():
    """A step in one coordinate of an fp32 operand, big enough to move its quantised value, moves
    sum(Y * dY) by the gradient times that value's move (the layer is linear in each operand)."""
    rng = np.random.default_rng(5)
    rows, nb, inn, out = 6, 2, 40, 24
    X, W = rng.standard_normal((rows, nb * inn)), rng.standard_normal((nb, out, inn))
    t = {k: dev(a, "f32")[0] for k, a in (("X", X), ("W", W), ("dY", rng.standard_normal((rows, nb * out))))}
    Wq, Xq = bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(t["X"], nblocks=nb)
    dX, dW, _ = bdl.mx4_linear_bwd(t["dY"], Xq, Wq)

    def loss(Xq, Wq):
        return float((bdl.mx4_linear_fwd(Xq, Wq, dtype="f32").double() * t["dY"].double()).sum())

    base, xv, wv = loss(Xq, Wq), bdl.mx4_dequantise(Xq), bdl.mx4_dequantise(Wq)
    for k in range(4):
        i, j = int(rng.integers(rows)), int(rng.integers(nb * inn))
        x2 = t["X"].clone()
        x2[i, j] = -x2[i, j] + 0.3
        q2 = bdl.mx4_quantise(x2, nblocks=nb)
        move = (bdl.mx4_dequantise(q2) - xv).double()
        assert abs(loss(q2, Wq) - base - float((dX.double() * move).sum())) < 1e-3
        w2 = t["W"].clone()
        w2[k % nb, i, j % inn] += 0.7
        q2 = bdl.mx4_quantise(w2)
        move = (bdl.mx4_dequantise(q2) - wv).double()
        assert abs(loss(Xq, q2) - base - float((dW.double() * move).sum())) < 1e-3


@pytest.mark.parametrize("rows,nb,inn,out", [(3, 2, 96, 80), (40, 2, 96, 80), (300, 2, 128, 192)])
def test_nan_and_infinity_stay_in_their_rows(rows, nb, inn, out):
    t, v = layer(rows, nb, inn, out, False, "bf16", seed=3)
    X, W = t["X"].clone(), t["W"].clone()
    X[1, inn + 5] = float("nan")     # row 1, block 1
    X[2, 3] = float("inf")           # row 2, block 0
    W[1, 7, 2] = float("inf")        # block 1, output 7
    Xq, Wq = bdl.mx4_quantise(X, nblocks=nb), bdl.mx4_quantise(W)
    bad = np.zeros((rows, nb, out), dtype=bool)
    bad[1, 1, :] = bad[2, 0, :] = bad[:, 1, 7] = True
    for Y in (bdl.mx4_linear_fwd(Xq, Wq), bdl.mx4_linear_fwd(X, Wq)):
        y = f64(Y).reshape(rows, nb, out)
        assert not np.isfinite(y[bad]).any()
        assert np.isfinite(y[~bad]).all()
    dX, dW, _ = bdl.mx4_linear_bwd(t["dY"], Xq, Wq)
    bad_x = np.zeros((rows, nb, inn), dtype=bool)
    bad_x[:, 1, :32] = True          # the NaN weight block's 32 inputs
    assert np.array_equal(np.isnan(f64(dX).reshape(rows, nb, inn)), bad_x)
    bad_w = np.zeros((nb, out, inn), dtype=bool)
    bad_w[1, :, :32] = bad_w[0, :, :32] = True   # columns of the NaN activation blocks (5 and 3 are in block 0 of 32)
    assert np.array_equal(np.isnan(f64(dW)), bad_w)


def drift(got, ref):
    """(normwise, signed) error of an fp32 tensor against a float64 one, both on the GPU."""
    d = got.double() - ref
    return float(d.norm() / ref.norm()), float((d * ref.sign()).sum() / ref.abs().sum())


# Sums of one sign, where cut-off additions all err the same way.  A run of 512 inputs is 32 additions of the leading
# part that may each cut off 2^-23 of the partial sum, which grows evenly: 16.5 * 2^-23 of the run.  The runs join with
# additions that are off by at most 2^-24 of a sum that grows as evenly.
def run_bound(k):
    return 16.5 * 2.0 ** -23 + (k / 512 / 2 + 1) * 2.0 ** -24


@pytest.mark.parametrize("rows,inn,out", [(8192, 8192, 512), (600, 8192, 8192), (300, 16384, 257), (16384, 1000, 300), (8192, 512, 2049)])
def test_fp32_sums_do_not_drift_with_their_length(rows, inn, out):
    g = torch.Generator(device="cuda").manual_seed(rows + inn)
    X, W, dY = (torch.rand(s, generator=g, device="cuda") + 0.01 for s in ((rows, inn), (1, out, inn), (rows, out)))
    Xq, Wq = bdl.mx4_quantise(X), bdl.mx4_quantise(W)
    x, w = bdl.mx4_dequantise(Xq).double(), bdl.mx4_dequantise(Wq)[0].double()
    dX, dW, db = bdl.mx4_linear_bwd(dY, Xq, Wq, bias=True)
    dy = dY.double()
    for got, ref, k, what in ((bdl.mx4_linear_fwd(X, Wq), X.double() @ w.T, inn, "Y"), (dX, dy @ w, out, "dX"), (dW[0], dy.T @ x, rows, "dW"),
                              (db, dy.sum(0), rows, "dbias"), (bdl.mx4_linear_fwd(X[:20].contiguous(), Wq), X[:20].double() @ w.T, inn, "Y of 20 rows")):
        norm, signed = drift(got, ref)
        assert norm <= run_bound(k) and abs(signed) <= run_bound(k), (what, k, norm, signed, run_bound(k))
    assert bdl.last_device_status() == 0


@pytest.mark.parametrize("rows,inn,out,bias", [(260, 65536, 257, True), (300, 262144, 132, False), (129, 16385, 1001, True)])
def test_fp32_results_of_two_quantised_operands_do_not_drift(rows, inn, out, bias):
    """Steps of 64 inputs that may each cut off 2^-23 of a sum that grows evenly, in runs of 4096."""
    g = torch.Generator(device="cuda").manual_seed(inn)
    X, W = (torch.rand(s, generator=g, device="cuda") + 0.01 for s in ((rows, inn), (1, out, inn)))
    # a scale of its own for every 32, so that sums are not whole numbers of a common step
    X *= torch.exp(torch.randn((rows, -(-inn // 32)), generator=g, device="cuda")).repeat_interleave(32, 1)[:, :inn]
    W *= torch.exp(torch.randn((1, out, -(-inn // 32)), generator=g, device="cuda")).repeat_interleave(32, 2)[:, :, :inn]
    b = torch.randn(out, generator=g, device="cuda") if bias else None
    Xq, Wq = bdl.mx4_quantise(X), bdl.mx4_quantise(W)
    ref = bdl.mx4_dequantise(Xq).double() @ bdl.mx4_dequantise(Wq)[0].double().T + (b.double() if bias else 0)
    Y = bdl.mx4_linear_fwd(Xq, Wq, bias=b)
    bound = 65 / 2 * 2.0 ** -23 + (inn / 4096 / 2 + 1) * 2.0 ** -24
    norm, signed = drift(Y, ref)
    assert norm <= bound and abs(signed) <= bound and bdl.last_device_status() == 0, (norm, signed, bound)
    assert torch.equal(Y, bdl.mx4_linear_fwd(Xq, Wq, bias=b))


def test_bf16_sums_of_a_very_long_batch_do_not_drift():
    """dW over 262144 rows of one sign: the mean error of 64 x 64 results is a mean of roundings, plus what runs of 4096
    rows cut off (256 additions, as above)."""
    rows, n = 1 << 18, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.rand((rows, n), generator=g, device="cuda", dtype=torch.bfloat16)
    Xq = bdl.mx4_quantise(X)
    x = bdl.mx4_dequantise(Xq)[:, :64].double()
    dY = X * torch.exp2(torch.arange(n, device="cuda") / 64).bfloat16()   # results spread over a bf16 binade
    dY[:, n // 2:] = X[:, :n // 2]
    Wq = bdl.mx4_quantise(torch.ones((1, n, n), device="cuda", dtype=torch.bfloat16))
    _, dW, _ = bdl.mx4_linear_bwd(dY, Xq, Wq, need_dX=False)
    ref = dY[:, :64].double().T @ x
    d = (dW[0, :64, :64].double() - ref) / ref
    assert float(d.abs().max()) <= 2.0 ** -8 + 128.5 * 2.0 ** -23 + 2.0 ** -17
    # a rounding to bf16 is off by at most 2^-8 / 2 of the value on average 0: five deviations of 4096 such
    assert abs(float(d.mean())) <= 128.5 * 2.0 ** -23 + 64 / 2 * 2.0 ** -24 + 5 * 2.0 ** -8 / 3 ** 0.5 / 64


@pytest.mark.parametrize("bits", [0x7f800001, -0x7fffff, 0x7f80ffff, 0x7fc00000])
@pytest.mark.parametrize("rows,nb,inn,out", [(3, 1, 70, 40), (24, 1, 4096, 2048), (200, 2, 256, 300)])
def test_nan_payloads_in_the_low_half_stay_nan(rows, nb, inn, out, bits):
    """fp32 operands are cut into bf16 parts: a NaN with nothing in its upper 16 bits but the exponent is one still."""
    rng = np.random.default_rng(4)
    X, dY = (dev(rng.standard_normal((rows, nb * n)), "f32")[0] for n in (inn, out))
    Wq = bdl.mx4_quantise(dev(rng.uniform(0.5, 1, (nb, out, inn)), "f32")[0])   # no zeros: infinities would stay
    Xq = bdl.mx4_quantise(dev(rng.uniform(0.5, 1, (rows, nb * inn)), "f32")[0], nblocks=nb)
    X.view(torch.int32)[1, 7] = bits
    dY.view(torch.int32)[2, 5] = bits
    Y = f64(bdl.mx4_linear_fwd(X, Wq)).reshape(rows, nb, out)
    bad = np.zeros(Y.shape, dtype=bool)
    bad[1, 0] = True
    assert np.array_equal(np.isnan(Y), bad) and np.isfinite(Y[~bad]).all()
    dX, dW, db = (f64(g) for g in bdl.mx4_linear_bwd(dY, Xq, Wq, bias=True))
    bad_x, bad_w, bad_b = np.zeros((rows, nb, inn), dtype=bool), np.zeros(dW.shape, dtype=bool), np.zeros(db.shape, dtype=bool)
    bad_x[2, 0], bad_w[0, 5], bad_b[5] = True, True, True
    for g, bad in ((dX.reshape(bad_x.shape), bad_x), (dW, bad_w), (db, bad_b)):
        assert np.array_equal(np.isnan(g), bad) and np.isfinite(g[~bad]).all()
    assert np.isnan(f64(bdl.mx4_dequantise(bdl.mx4_quantise(X, nblocks=nb)))[1, :min(32, inn)]).all()


def test_extreme_scales():
    """Weights of 2^100 and 2^-100 against activations that bring the products back into range."""
    rng = np.random.default_rng(9)
    inn, out = 64, 40
    for rows in (2, 150):
        X = rng.standard_normal((rows, inn))
        W = rng.standard_normal((1, out, inn))
        X[:, :32] *= 2.0 ** -100
        W[:, :, :32] *= 2.0 ** 100
        X[:, 32:] *= 2.0 ** 90
        W[:, :, 32:] *= 2.0 ** -90
        for dtype in ("bf16", "f32"):
            t, x = dev(X, dtype)
            w, wv = dev(W, dtype)
            v = dict(w=oracle.mx4_round(wv), b=None)
            Wq = bdl.mx4_quantise(w)
            check_forward(bdl.mx4_linear_fwd(t, Wq), x, v, inn, dtype, "weights only")
            check_forward(bdl.mx4_linear_fwd(bdl.mx4_quantise(t), Wq), oracle.mx4_round(x), v, inn, dtype, "both")


# ---------------------------------------------------------------- Monarch map
MONARCH = [  # (rows, nb1, in1, out1, nb2, in2, out2, out_transpose)
    (1, 4, 256, 256, 4, 256, 1024, 0), (3, 16, 16, 16, 16, 16, 16, 1), (1, 64, 64, 64, 64, 64, 64, 1),
    (32, 32, 32, 32, 32, 32, 32, 1), (33, 16, 48, 48, 48, 16, 64, 1), (7, 4, 250, 250, 4, 250, 1000, 0),
    (5, 3, 10, 8, 4, 6, 5, 1), (2, 1, 40, 24, 2, 12, 9, 0), (9, 2, 300, 129, 6, 43, 17, 1), (12, 5, 33, 70, 7, 50, 21, 0),
    (3, 2, 2048, 1100, 2, 1100, 1030, 0), (20, 8, 640, 640, 8, 640, 1024, 1), (64, 4, 256, 64, 4, 64, 64, 0), (65, 8, 64, 64, 8, 64, 128, 0),
    (200, 32, 32, 32, 32, 32, 32, 1), (300, 4, 256, 256, 4, 256, 1024, 0), (17, 13, 40, 26, 13, 26, 9, 1),
    (33, 52, 52, 52, 52, 52, 52, 1), (300, 4, 256, 256, 4, 256, 256, 0), (600, 3, 10, 8, 4, 6, 5, 1), (500, 2, 300, 129, 6, 43, 17, 1),
    (1200, 32, 32, 32, 32, 32, 32, 1), (10, 9, 100, 33, 27, 11, 6, 1), (64, 64, 64, 64, 64, 64, 64, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nb1,in1,out1,nb2,in2,out2,tr", MONARCH)
def test_monarch_forward(rows, nb1, in1, out1, nb2, in2, out2, tr, dtype):
    shape = dict(nb1=nb1, in1=in1, out1=out1, nb2=nb2, in2=in2, out2=out2, out_transpose=tr)
    rng = np.random.default_rng(rows + in1 + out2)
    X, x = dev(rng.standard_normal((rows, nb1 * in1)), dtype)
    R, r = dev(rng.uniform(-1, 1, (nb1, out1, in1)) / np.sqrt(in1), dtype)
    L, l = dev(rng.uniform(-1, 1, (nb2, out2, in2)) / np.sqrt(in2), dtype)
    Rq, Lq = bdl.mx4_quantise(R), bdl.mx4_quantise(L)
    Y = bdl.mx4_fwd(X, Rq, Lq, shape)
    assert bdl.last_device_status() == 0
    r, l = oracle.mx4_round(r), oracle.mx4_round(l)
    ref = oracle.forward(shape, x, r, l)
    mags = oracle.forward(shape, np.abs(x), np.abs(r), np.abs(l))
    # long batches hold the middle vector in the tensors' type: half a step of every middle value
    middle = HALF[dtype] * 1.01 * oracle.forward(shape, np.abs(x), np.abs(r), np.abs(l))
    close(Y, ref, mags, in1 + in2 + 4, dtype, "Y", extra=middle)
    assert torch.equal(Y, bdl.mx4_fwd(X, Rq, Lq, shape))


def test_monarch_few_tokens_keep_the_middle_vector():
    """Up to 64 tokens the middle vector is not rounded to bf16: the result is half a step off."""
    shape = dict(nb1=32, in1=32, out1=32, nb2=32, in2=32, out2=32, out_transpose=1)
    rng = np.random.default_rng(1)
    R, r = dev(rng.uniform(-1, 1, (32, 32, 32)), "bf16")
    L, l = dev(rng.uniform(-1, 1, (32, 32, 32)), "bf16")
    r, l = oracle.mx4_round(r), oracle.mx4_round(l)
    for rows in (1, 4, 17, 64):
        X, x = dev(rng.standard_normal((rows, 1024)), "bf16")
        Y = bdl.mx4_fwd(X, bdl.mx4_quantise(R), bdl.mx4_quantise(L), shape)
        mags = oracle.forward(shape, np.abs(x), np.abs(r), np.abs(l))
        # the middle value may be split into two bf16 parts: 2^-16 of it is lost at most
        close(Y, oracle.forward(shape, x, r, l), mags, 70, "bf16", "Y", extra=2.0 ** -16 * mags)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,inn,mid,out", [(1, 4, 2, 3), (8, 40, 64, 130), (20, 33, 250, 70), (64, 64, 1024, 2048), (24, 64, 1024, 2048)])
def test_monarch_few_tokens_keep_every_bit_of_the_middle_vector(rows, inn, mid, out, dtype):
    """Middle values of 24 one bits, and beside each the negative of its first 16: the result is the last
    eight, and every sum on the way to it is exact in fp32."""
    ones = 255 * np.exp2([-7.0, -15.0, -23.0])
    X, R, L = np.zeros((rows, inn)), np.zeros((1, mid, inn)), np.zeros((1, out, mid))
    X[:, :3] = ones * np.exp2(np.arange(rows) % 5)[:, None]
    R[0, 0::2, :3], R[0, 1::2, :2] = 1, -1
    for o in range(out):
        at = 2 * (o % (mid // 2))
        L[0, o, at:at + 2] = 1
    shape = dict(nb1=1, in1=inn, out1=mid, nb2=1, in2=mid, out2=out, out_transpose=0)
    t = [dev(a, dtype)[0] for a in (X, R, L)]
    Y = bdl.mx4_fwd(t[0], bdl.mx4_quantise(t[1]), bdl.mx4_quantise(t[2]), shape)
    assert np.array_equal(f64(Y), np.repeat(X[:, 2:3], out, axis=1))


@pytest.mark.parametrize("rows", [1, 4, 17, 64])
def test_monarch_few_tokens_are_rounded_once(rows):
    """Both sums are fp32 sums of the middle vector's full values: no more than their own rounding on top of half
    a step of the bf16 result."""
    for shape in (dict(nb1=32, in1=32, out1=32, nb2=32, in2=32, out2=32, out_transpose=1),
                  dict(nb1=4, in1=256, out1=256, nb2=4, in2=256, out2=1024, out_transpose=0)):
        rng = np.random.default_rng(rows)
        X, x = dev(rng.standard_normal((rows, 1024)), "bf16")
        R, r = dev(rng.uniform(-1, 1, (shape["nb1"], shape["out1"], shape["in1"])), "bf16")
        L, l = dev(rng.uniform(-1, 1, (shape["nb2"], shape["out2"], shape["in2"])), "bf16")
        Y = bdl.mx4_fwd(X, bdl.mx4_quantise(R), bdl.mx4_quantise(L), shape)
        r, l = oracle.mx4_round(r), oracle.mx4_round(l)
        mags = oracle.forward(shape, np.abs(x), np.abs(r), np.abs(l))
        # runs of 32 inputs (two steps that cut off, at most 2^-23 each), then one rounded addition a run
        terms = sum(2 * 3 + n / 32 for n in (shape["in1"], shape["in2"])) + 2
        close(Y, oracle.forward(shape, x, r, l), mags, terms, "bf16", "Y")


@pytest.mark.parametrize("rows,mid", [(524281, 60000), (524289, 24), (65537, 24), (131072, 40)])
def test_monarch_rows_beyond_one_launch(rows, mid):
    """The first and last rows of every pass of 65536, as if they had come alone; nothing behind the last."""
    shape = dict(nb1=1, in1=8, out1=mid, nb2=1, in2=mid, out2=8, out_transpose=0)
    g = torch.Generator(device="cuda").manual_seed(mid)
    R, L = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((1, mid, 8), (1, 8, mid)))
    Rq, Lq = bdl.mx4_quantise(R), bdl.mx4_quantise(L)
    X = torch.randn((rows, 8), generator=g, device="cuda").bfloat16()
    Y, ok = guarded((rows, 8), torch.bfloat16)
    bdl.mx4_fwd(X, Rq, Lq, shape, Y=Y)
    assert ok() and bdl.last_device_status() == 0
    at = torch.tensor([r for p in range(0, rows, 65536) for r in (p, min(p + 65535, rows - 1))], device="cuda")
    r, l = oracle.mx4_round(f64(R)), oracle.mx4_round(f64(L))
    x = f64(X[at])
    ref, mags = oracle.forward(shape, x, r, l), oracle.forward(shape, np.abs(x), np.abs(r), np.abs(l))
    close(Y[at], ref, mags, 8 + mid / 32 + 8, "bf16", "Y")
    assert bool(torch.isfinite(Y).all()) and float((Y.abs().sum(1) == 0).sum()) == 0


# ---------------------------------------------------------------- as they are used
def test_training_steps_of_a_quantised_layer():
    """Forward, backward and update of fp32 master weights for three steps: every step's outputs are the
    oracle's for that step's weights."""
    rows, nb, inn, out = 150, 2, 128, 192
    rng = np.random.default_rng(11)
    W = torch.from_numpy(rng.uniform(-1, 1, (nb, out, inn)) / np.sqrt(inn)).float().cuda()
    b = torch.zeros(nb * out, device="cuda")
    for step in range(3):
        X, x = dev(rng.standard_normal((rows, nb * inn)), "bf16")
        T, target = dev(rng.standard_normal((rows, nb * out)), "bf16")
        Wq, Xq = bdl.mx4_quantise(W), bdl.mx4_quantise(X, nblocks=nb)
        bias, bv = dev(f64(b), "bf16")
        Y = bdl.mx4_linear_fwd(Xq, Wq, bias=bias, dtype="bf16")
        v = dict(w=oracle.mx4_round(f64(W)), b=bv)
        xr = oracle.mx4_round(x.reshape(rows, nb, inn)).reshape(rows, -1)
        check_forward(Y, xr, v, inn, "bf16", "Y")
        dY = (Y - T) / rows
        dX, dW, db = bdl.mx4_linear_bwd(dY, Xq, Wq, bias=True)
        refs = oracle.mx4_linear_backward(f64(dY), xr, v["w"])
        mags = oracle.mx4_linear_backward(np.abs(f64(dY)), np.abs(xr), np.abs(v["w"]))
        for g, r, m, terms, what in zip((dX, dW, db), refs, mags, (out, rows, rows), ("dX", "dW", "db")):
            close(g, r, m, terms + 2, "bf16", what)
        W -= 0.5 * dW.float()
        b -= 0.5 * db.float()
    assert bdl.last_device_status() == 0


def test_serving_chain_matches_its_parts():
    """Prompt, then single tokens, through an MX4 layer and an MX4 Monarch map: a token's result does not
    depend on the batch it came in beyond the two kernels' rounding."""
    rng = np.random.default_rng(12)
    shape = dict(nb1=16, in1=32, out1=32, nb2=16, in2=32, out2=32, out_transpose=0)
    W, _ = dev(rng.uniform(-1, 1, (1, 512, 512)) / 22, "bf16")
    R, _ = dev(rng.uniform(-1, 1, (16, 32, 32)) / 5, "bf16")
    Wq, Rq = bdl.mx4_quantise(W), bdl.mx4_quantise(R)
    X, _ = dev(rng.standard_normal((300, 512)), "bf16")
    H = bdl.mx4_linear_fwd(X, Wq)
    Y = bdl.mx4_fwd(H, Rq, Rq, shape)
    for r in (0, 1, 150, 299):
        h = bdl.mx4_linear_fwd(X[r:r + 1], Wq)
        assert float((h - H[r:r + 1]).abs().max()) <= 2.0 ** -7 * float(H[r].abs().max())
        y = bdl.mx4_fwd(H[r:r + 1].contiguous(), Rq, Rq, shape)
        assert float((y - Y[r:r + 1]).float().norm()) <= 2.0 ** -6 * float(Y[r].float().norm())


@pytest.mark.parametrize("tr", [0, 1])
@pytest.mark.parametrize("blocks", [64, 32])
def test_factors_that_a_product_has_just_written(blocks, tr):
    """Monarch factors that are the result of the call before (a layer that makes another's weights): the maps that read
    them wait for it.  New factors each time, so that old ones would show."""
    n = blocks * blocks
    shape = dict(nb1=blocks, in1=blocks, out1=blocks, nb2=blocks, in2=blocks, out2=blocks, out_transpose=tr)
    g = torch.Generator(device="cuda").manual_seed(blocks)
    Wq = bdl.mx4_quantise(torch.randn((1, n, 4096), generator=g, device="cuda").bfloat16() / 500)
    X, dY = (torch.randn((500, n), generator=g, device="cuda").bfloat16() for _ in range(2))
    R, L = (torch.empty((blocks, n), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Xs = [torch.randn((blocks, 4096), generator=g, device="cuda").bfloat16() for _ in range(6)]

    def run(k, wait):
        bdl.mx4_linear_fwd(Xs[k], Wq, Y=L)
        bdl.mx4_linear_fwd(Xs[k + 1], Wq, Y=R)
        if wait:
            torch.cuda.synchronize()
        f = R.view(blocks, blocks, blocks), L.view(blocks, blocks, blocks)
        if k % 2:
            return [bdl.fwd(X, *f, shape), bdl.fwd_ws(X, *f, shape)]
        return list(bdl.bwd(dY, X, *f, shape))
    want = [run(k, True) for k in range(5)]
    for _ in range(3):
        for k in (0, 4, 1, 2, 3):
            assert all(torch.equal(a, b) for a, b in zip(run(k, False), want[k])), k


def guarded(shape, dtype):
    """A tensor inside a larger buffer filled with a pattern, and a check that the rest is untouched."""
    n = int(np.prod(shape))
    pad = 256
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    view = buf[pad:pad + n].view(shape)

    def intact():
        return bool((buf[:pad] == 7).all() and (buf[pad + n:] == 7).all())
    return view, intact


@pytest.mark.parametrize("rows,nb,inn,out", [(1, 1, 33, 130), (9, 3, 40, 24), (130, 2, 96, 200), (257, 1, 256, 72), (65, 2, 64, 64)])
def test_nothing_is_written_outside_the_outputs(rows, nb, inn, out):
    t, _ = layer(rows, nb, inn, out, True, "bf16", seed=4)
    Wq, Xq = bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(t["X"], nblocks=nb)
    for X in (t["X"], Xq):
        Y, ok = guarded((rows, nb * out), torch.bfloat16)
        want = bdl.mx4_linear_fwd(X, Wq, bias=t["b"])
        assert torch.equal(bdl.mx4_linear_fwd(X, Wq, bias=t["b"], Y=Y), want) and ok()
    dX, ok1 = guarded((rows, nb * inn), torch.bfloat16)
    dW, ok2 = guarded((nb, out, inn), torch.bfloat16)
    db, ok3 = guarded((nb * out,), torch.bfloat16)
    want = bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=True)
    need = bdl.mx4_linear_workspace_bytes(rows, nb, inn, out, "bf16", True, backward=True)
    ws = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
    got = bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=True, dX=dX, dW=dW, dbias=db, workspace=ws[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and ok1() and ok2() and ok3()
    assert bool((ws[need:] == 9).all())
    out_v, ok = guarded((rows, nb * inn), torch.bfloat16)
    bdl.mx4_dequantise(Xq, "bf16", out=out_v)
    assert ok()


def test_no_rows():
    W, _ = dev(np.ones((2, 40, 64)), "bf16")
    Wq = bdl.mx4_quantise(W)
    X = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    Xq = bdl.mx4_quantise(X, nblocks=2)
    assert bdl.mx4_dequantise(Xq).shape == (0, 128)
    assert bdl.mx4_linear_fwd(X, Wq).shape == (0, 80) and bdl.mx4_linear_fwd(Xq, Wq).shape == (0, 80)
    dX, dW, db = bdl.mx4_linear_bwd(torch.empty(0, 80, dtype=torch.bfloat16, device="cuda"), Xq, Wq, bias=True)
    assert dX.shape == (0, 128) and not dW.any() and not db.any()
    shape = dict(nb1=2, in1=64, out1=40, nb2=2, in2=40, out2=8, out_transpose=1)
    assert bdl.mx4_fwd(X, Wq, bdl.mx4_quantise(torch.ones(2, 8, 40, dtype=torch.bfloat16, device="cuda")), shape).shape == (0, 16)


def everything(t, Wq, Rq, shape, nb, stream=None):
    Xq = bdl.mx4_quantise(t["X"], nblocks=nb, stream=stream)
    out = [bdl.mx4_dequantise(Xq, stream=stream), bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"], stream=stream),
           bdl.mx4_linear_fwd(t["X"], Wq, bias=t["b"], stream=stream), bdl.mx4_fwd(t["X"], Rq, Rq, shape, stream=stream)]
    return out + list(bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=True, stream=stream))


@pytest.mark.parametrize("rows", [2, 40, 260])
def test_captured_graphs_and_streams(rows):
    """Two graphs of the whole set replayed on two streams at once, new inputs in place, and a call given
    a stream: all as the plain calls on those inputs."""
    nb, inn, out = 4, 64, 96
    shape = dict(nb1=4, in1=64, out1=64, nb2=4, in2=64, out2=64, out_transpose=0)
    sets, graphs, outs = [], [], []
    for k in range(2):
        t, _ = layer(rows, nb, inn, out, True, "bf16", seed=20 + k)
        R, _ = dev(np.random.default_rng(k).uniform(-1, 1, (4, 64, 64)), "bf16")
        sets.append((t, bdl.mx4_quantise(t["W"]), bdl.mx4_quantise(R), shape, nb))
    everything(*sets[0])
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(*s))
        graphs.append(g)
    new = [layer(rows, nb, inn, out, True, "bf16", seed=30 + k)[0] for k in range(2)]
    for s, n in zip(sets, new):
        for k in ("X", "dY", "b"):
            s[0][k].copy_(n[k])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        plain = everything(*s)
        assert all(torch.equal(a, b) for a, b in zip(o, plain))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        given = everything(*s, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(given, plain))
    assert bdl.last_device_status() == 0


def test_large_offsets():
    """A tensor whose codes pass 2^31 elements: the last rows are rounded and read where they belong."""
    rows, cols = 1 << 19, 4100
    X = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    tail, v = dev(rng.standard_normal((3, cols)), "bf16")
    X[-3:] = tail
    q = bdl.mx4_quantise(X)
    del X
    W, wv = dev(rng.uniform(-1, 1, (1, 8, cols)) / 64, "bf16")
    Y = bdl.mx4_linear_fwd(q, bdl.mx4_quantise(W))
    assert not Y[:-3].any()
    ref = oracle.mx4_linear_forward(oracle.mx4_round(v), oracle.mx4_round(wv))
    mags = oracle.mx4_linear_forward(np.abs(oracle.mx4_round(v)), np.abs(oracle.mx4_round(wv)))
    close(Y[-3:], ref, mags, cols + 2, "bf16", "Y")
    back = bdl.mx4_dequantise(q)
    assert np.array_equal(f64(back[-3:]), oracle.mx4_round(v)) and not back[:16].any()


def test_a_copied_weight_outlives_the_first():
    import copy
    t, v = layer(5, 2, 96, 64, False, "bf16")
    Wq = bdl.mx4_quantise(t["W"])
    want = bdl.mx4_linear_fwd(t["X"], Wq)
    twin = copy.deepcopy(Wq)
    Wq.codes.zero_()
    assert torch.equal(bdl.mx4_linear_fwd(t["X"], twin), want)
    check_forward(want, v["x"], v, 96, "bf16", "Y")


def test_two_threads_on_their_own_streams():
    import threading
    t, _ = layer(700, 2, 400, 512, True, "bf16")
    Wq = bdl.mx4_quantise(t["W"])
    shape = dict(nb1=16, in1=16, out1=16, nb2=16, in2=16, out2=16, out_transpose=1)
    Rq = bdl.mx4_quantise(torch.randn(16, 16, 16, device="cuda").bfloat16())

    def work(k):
        X, dY = t["X"] * 2.0 ** k, t["dY"] * 2.0 ** -k
        Xq = bdl.mx4_quantise(X, nblocks=2)
        return [bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"]), bdl.mx4_linear_fwd(X, Wq), bdl.mx4_linear_fwd(X[:1 + k], Wq, bias=t["b"]),
                *bdl.mx4_linear_bwd(dY, Xq, Wq, bias=True), bdl.mx4_fwd(X[:3, :256].contiguous(), Rq, Rq, shape)]
    want = [work(k) for k in range(2)]
    torch.cuda.synchronize()
    faults = []

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = work(k)
                    if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                        faults.append(k)
        except Exception as e:  # noqa: BLE001 - reported below
            faults.append(e)
    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not faults and bdl.last_device_status() == 0


# ---------------------------------------------------------------- every kernel by its path
# Sizes for each kernel of a product, with the path they have to take: full and ragged tiles, fewer rows than a tile, result rows
# that TMA can and cannot store, several tiles a CTA.  (product, rows, nblocks, in, out, dtype, path)
PATHS = [
    ("both", 777, 1, 96, 250, "bf16", 2), ("both", 33, 5, 200, 500, "bf16", 2), ("both", 127, 2, 96, 777, "f32", 2), ("both", 2000, 9, 300, 60, "f32", 2),
    ("both", 1300, 5, 96, 130, "bf16", 3), ("both", 9, 5, 200, 2050, "bf16", 3), ("both", 127, 5, 200, 2000, "f32", 3),
    ("both", 777, 3, 200, 500, "bf16", 3), ("both", 1300, 5, 96, 130, "f32", 3), ("both", 3000, 5, 700, 128, "bf16", 3),
    ("both", 129, 5, 96, 2050, "bf16", 4), ("both", 520, 5, 96, 1000, "bf16", 4), ("both", 4000, 2, 96, 260, "f32", 4), ("both", 129, 5, 96, 2050, "f32", 4),
    ("both", 9, 5, 96, 4096, "bf16", 5), ("both", 129, 5, 96, 2000, "f32", 5),
    ("both", 2050, 5, 2048, 130, "bf16", 6), ("both", 3001, 1, 2000, 4001, "bf16", 6), ("both", 2500, 1, 4096, 2560, "bf16", 6), ("both", 2050, 5, 2048, 130, "f32", 6),
    ("both", 2500, 1, 2090, 4000, "f32", 6), ("both", 257, 1, 16390, 200, "f32", 7), ("both", 200, 1, 20000, 1001, "f32", 7),
    ("both", 9, 1, 16400, 4096, "f32", 7), ("both", 1300, 3, 16500, 1000, "f32", 7),
    ("weights", 9, 5, 4096, 260, "bf16", 1), ("weights", 16, 1, 4096, 4096, "bf16", 1), ("weights", 31, 5, 520, 2000, "bf16", 1), ("weights", 64, 1, 4000, 1000, "bf16", 1),
    ("weights", 50, 2, 2047, 2050, "bf16", 1), ("weights", 1, 1, 4096, 4096, "f32", 1), ("weights", 9, 1, 4095, 777, "f32", 1), ("weights", 32, 5, 520, 1000, "f32", 1),
    ("weights", 257, 5, 96, 500, "bf16", 8), ("weights", 65, 5, 100, 2000, "bf16", 8), ("weights", 777, 2, 96, 250, "f32", 8), ("weights", 33, 5, 97, 2050, "f32", 8),
    ("weights", 129, 5, 96, 2050, "bf16", 9), ("weights", 2000, 1, 1024, 4096, "bf16", 9), ("weights", 2001, 1, 1000, 4001, "bf16", 9),
    ("weights", 129, 5, 96, 2050, "f32", 9), ("weights", 2001, 1, 1001, 4000, "f32", 9),
    ("weights", 300, 1, 2048, 130, "bf16", 24), ("weights", 100, 5, 2048, 72, "bf16", 24), ("weights", 300, 2, 520, 130, "f32", 24), ("weights", 33, 1, 521, 2000, "f32", 24),
    ("weights", 129, 5, 4096, 130, "bf16", 25), ("weights", 257, 1, 4096, 1000, "bf16", 25), ("weights", 129, 5, 1000, 130, "f32", 25), ("weights", 129, 1, 4096, 260, "f32", 25),
    ("dX", 129, 5, 2048, 72, "bf16", 9), ("dX", 2500, 1, 1024, 4096, "bf16", 9), ("dX", 1500, 2, 1001, 2050, "bf16", 9), ("dX", 129, 5, 2048, 72, "f32", 9),
    ("dX", 129, 1, 96, 2000, "bf16", 24), ("dX", 9, 1, 97, 2000, "bf16", 24), ("dX", 129, 1, 97, 500, "f32", 24),
    ("dX", 129, 5, 200, 4096, "bf16", 25), ("dX", 129, 5, 201, 1000, "f32", 25),
    ("dW", 129, 5, 2048, 130, "bf16", 9), ("dW", 2000, 1, 1024, 4000, "bf16", 9), ("dW", 1501, 2, 1000, 2050, "bf16", 9), ("dW", 9, 5, 2047, 130, "f32", 9),
    ("dW", 1300, 1, 96, 72, "bf16", 24), ("dW", 520, 1, 97, 72, "f32", 24), ("dW", 4000, 5, 200, 130, "bf16", 25), ("dW", 2050, 1, 521, 130, "f32", 25),
]


def gpu_layer(rows, nb, inn, out, dtype, seed, x_by=1.0, w_by=1.0):
    """Tensors of a layer made on the GPU, its quantised operands, and every operand's values in 64 bits there (roundings to
    MX4 are compared with the oracle above, so a quantised operand's values are what it dequantises to)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * rows + inn + out)
    T = TORCH[dtype]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    t = {"X": (normal(rows, nb * inn) * x_by).to(T), "W": (normal(nb, out, inn) * w_by / inn ** 0.5).to(T),
         "dY": normal(rows, nb * out).to(T), "b": normal(nb * out).to(T)}
    Xq, Wq = bdl.mx4_quantise(t["X"], nblocks=nb), bdl.mx4_quantise(t["W"])
    v = {k: t[k].double() for k in ("X", "dY", "b")}
    v["Xq"], v["W"] = bdl.mx4_dequantise(Xq).double(), bdl.mx4_dequantise(Wq).double()
    return t, Xq, Wq, v


def gpu_product(product, v, nb, absolute=False):
    v = {k: x.abs() for k, x in v.items()} if absolute else v
    dy, w = v["dY"].view(len(v["dY"]), nb, -1).transpose(0, 1), v["W"]
    x = v["X" if product == "weights" else "Xq"].view(len(v["X"]), nb, -1).transpose(0, 1)
    if product in ("both", "weights"):
        return (x @ w.transpose(1, 2)).transpose(0, 1).reshape(len(v["X"]), -1) + v["b"]
    return (dy @ w).transpose(0, 1).reshape(len(v["X"]), -1) if product == "dX" else dy.transpose(1, 2) @ x


def gpu_close(product, got, v, nb, terms, dtype):
    ref, mags = gpu_product(product, v, nb), gpu_product(product, v, nb, True)
    off = (got.double() - ref).abs() - (HALF[dtype] * ref.abs() + (terms * 2.0 ** -23) * mags + 2.0 ** -126)
    assert got.shape == ref.shape and bool((off <= 0).all()), (product, int((~(off <= 0)).sum()), off.max())


@pytest.mark.parametrize("product,rows,nb,inn,out,dtype,path", PATHS)
def test_every_kernel(product, rows, nb, inn, out, dtype, path):
    assert bdl.mx4_linear_path(product, rows, nb, inn, out, dtype) == path
    t, Xq, Wq, v = gpu_layer(rows, nb, inn, out, dtype, 8)
    if product in ("both", "weights"):
        got, ok = guarded((rows, nb * out), TORCH[dtype])
        bdl.mx4_linear_fwd(Xq if product == "both" else t["X"], Wq, bias=t["b"], Y=got)
    else:
        got, ok = guarded((rows, nb * inn) if product == "dX" else (nb, out, inn), TORCH[dtype])
        bdl.mx4_linear_bwd(t["dY"], Xq if product == "dW" else None, Wq, need_dX=product == "dX", **{product: got})
    gpu_close(product, got, v, nb, {"dX": out, "dW": rows}.get(product, inn) + 2, dtype)
    assert ok() and bdl.last_device_status() == 0


# a few-row call and a long one of the same layer, on every path of the two forwards that has no such test above
@pytest.mark.parametrize("rows,nb,inn,out,both,weights", [
    (16, 2, 1024, 4096, 2, 1), (900, 2, 600, 1024, 3, 8), (700, 2, 1024, 2050, 4, 9), (1500, 2, 600, 1024, 5, 9), (2100, 2, 2048, 1030, 6, 9)])
def test_nan_and_infinity_stay_in_their_rows_on_every_path(rows, nb, inn, out, both, weights):
    assert bdl.mx4_linear_path("both", rows, nb, inn, out) == both
    assert bdl.mx4_linear_path("weights", rows, nb, inn, out) == weights
    test_nan_and_infinity_stay_in_their_rows(rows, nb, inn, out)


@pytest.mark.parametrize("rows,nb,inn,out,both,weights", [
    (16, 1, 2048, 4096, 2, 1), (2100, 2, 2048, 1030, 6, 9), (1500, 2, 600, 1024, 5, 9), (777, 3, 200, 500, 3, 8), (1025, 1, 700, 4001, 4, 8)])
def test_nothing_is_written_outside_the_outputs_on_every_path(rows, nb, inn, out, both, weights):
    assert bdl.mx4_linear_path("both", rows, nb, inn, out) == both
    assert bdl.mx4_linear_path("weights", rows, nb, inn, out) == weights
    test_nothing_is_written_outside_the_outputs(rows, nb, inn, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,out,both", [(520, 1024, 2), (1300, 1024, 3), (3000, 1030, 4), (1300, 2000, 5), (3000, 4001, 6)])
def test_extreme_scales_on_every_path(rows, out, both, dtype):
    """Weights of 2^100 and 2^-100 against activations that bring the products back into range, in tensor-core tiles."""
    inn = 2112 if both == 6 else 544
    assert bdl.mx4_linear_path("both", rows, 1, inn, out, dtype) == both
    up = torch.where(torch.arange(inn, device="cuda") // 32 % 2 == 0, 100.0, -90.0)
    t, Xq, Wq, v = gpu_layer(rows, 1, inn, out, dtype, 9, torch.exp2(-up), torch.exp2(up))
    dX, dW, _ = bdl.mx4_linear_bwd(t["dY"], Xq, Wq)
    for product, got, terms in (("both", bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"]), inn), ("weights", bdl.mx4_linear_fwd(t["X"], Wq, bias=t["b"]), inn),
                                ("dX", dX, out), ("dW", dW, rows)):
        gpu_close(product, got, v, 1, terms + 2, dtype)


@pytest.mark.parametrize("rows,nb,inn,out,dtype", [(16, 1, 4096, 4096, "bf16"), (2100, 1, 2048, 1030, "bf16"), (900, 2, 1100, 1024, "f32")])
def test_captured_graphs_of_long_layers(rows, nb, inn, out, dtype):
    """Two graphs of a layer's step, with memory of their own, replayed at once on two streams and new inputs."""
    def step(t, Wq):
        Xq = bdl.mx4_quantise(t["X"], nblocks=nb)
        return [bdl.mx4_linear_fwd(Xq, Wq, bias=t["b"]), bdl.mx4_linear_fwd(t["X"], Wq, bias=t["b"]),
                *bdl.mx4_linear_bwd(t["dY"], Xq, Wq, bias=True)]
    sets, graphs, outs = [], [], []
    for k in range(2):
        t = gpu_layer(rows, nb, inn, out, dtype, 40 + k)[0]
        sets.append((t, bdl.mx4_quantise(t["W"])))
        step(*sets[k])
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    for k, s in enumerate(sets):
        n = gpu_layer(rows, nb, inn, out, dtype, 50 + k)[0]
        for key in ("X", "dY", "b"):
            s[0][key].copy_(n[key])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        assert all(torch.equal(a, b) for a, b in zip(o, step(*s)))
    assert bdl.last_device_status() == 0


@pytest.mark.parametrize("rows,nb1,in1,out1,nb2,in2,out2,tr,dtype,path", [
    (3000, 32, 32, 32, 32, 32, 32, 1, "bf16", 2), (2000, 16, 48, 48, 48, 16, 64, 1, "bf16", 3), (700, 64, 64, 64, 64, 64, 64, 1, "bf16", 4),
    (1500, 4, 256, 256, 4, 256, 1024, 0, "bf16", 1), (1500, 4, 256, 256, 4, 256, 256, 0, "bf16", 0), (3000, 32, 32, 32, 32, 32, 32, 1, "f32", 0),
    (700, 64, 64, 64, 64, 64, 64, 1, "f32", 0), (70, 2, 1024, 1000, 2, 1000, 1024, 0, "bf16", 0), (70, 2, 1024, 1000, 2, 1000, 1024, 0, "f32", 0)])
def test_monarch_forward_of_a_prompt(rows, nb1, in1, out1, nb2, in2, out2, tr, dtype, path):
    shape = dict(nb1=nb1, in1=in1, out1=out1, nb2=nb2, in2=in2, out2=out2, out_transpose=tr)
    assert bdl.mx4_fwd_path(shape, rows, dtype) == path and bdl.mx4_fwd_path(shape, 64, dtype) == 0
    test_monarch_forward(rows, nb1, in1, out1, nb2, in2, out2, tr, dtype)
