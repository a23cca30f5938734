"""Cases of the microscaled 4-bit (MX4) operators and what each of them computes.

MX4: 32 neighbouring values along a product's inner axis share one power-of-two scale
2^(floor(log2(largest magnitude)) - 2), and each is held in 4 bits (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6
with a sign), rounded to the nearest of those (ties to the even code) and cut at 6.

  quantise   a tensor to MX4 and back to its values
  linear     block-diagonal linear layer, X (quantised in the call) and W both in MX4
  weights    the same layer with X as it is and W in MX4 (serving; one token upwards)
  monarch    the Monarch map with both factors in MX4 (serving; few tokens)
  backward   gradients of `linear` for the rounded operands: dX, dW and dbias

`run` computes the plain form with elementary torch operations where `own` is false and calls the
framework where it is true.
"""
import math
import random

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # activations of a long batch ahead of a four-block layer
        dict(name="quantise_activations", op="quantise", weights=False, rows=16384, nblocks=4, cols=1024, dtype="bf16"),
        # master weights of a small layer whose sizes are no multiples of the scale block
        dict(name="quantise_weights_odd", op="quantise", weights=True, rows=333, nblocks=5, cols=1000, dtype="f32"),
        # a dense 4096 -> 4096 layer over a long batch
        dict(name="linear_dense", op="linear", rows=8192, nblocks=1, in_blk=4096, out_blk=4096, bias=False, dtype="bf16"),
        # the wide factor of the four-block 1024 -> 4096 layer at its 10000 rows
        dict(name="linear_four_blocks", op="linear", rows=10000, nblocks=4, in_blk=256, out_blk=1024, bias=True, dtype="bf16"),
        # a ragged batch and odd block sizes
        dict(name="linear_odd", op="linear", rows=777, nblocks=3, in_blk=200, out_blk=500, bias=True, dtype="bf16"),
        # one token through a dense layer while decoding
        dict(name="weights_one_token", op="weights", rows=1, nblocks=1, in_blk=4096, out_blk=4096, bias=True, dtype="bf16"),
        # a small decoding batch through the blocks of a padded four-block layer (1000 -> 4000)
        dict(name="weights_batch_odd", op="weights", rows=33, nblocks=4, in_blk=250, out_blk=1000, bias=False, dtype="bf16"),
        # a prompt's tokens
        dict(name="weights_prompt", op="weights", rows=2000, nblocks=1, in_blk=1024, out_blk=4096, bias=True, dtype="bf16"),
        # one token through the four-block 1024 -> 4096 Monarch layer
        dict(name="monarch_one_token", op="monarch", rows=1, nb1=4, in1=256, out1=256, nb2=4, in2=256, out2=1024,
             out_transpose=0, dtype="bf16"),
        # a decoding batch through the square n = 4096 map
        dict(name="monarch_batch", op="monarch", rows=32, nb1=64, in1=64, out1=64, nb2=64, in2=64, out2=64,
             out_transpose=1, dtype="bf16"),
        # a training step's backward of a dense 1024 -> 4096 layer
        dict(name="backward_dense", op="backward", rows=8192, nblocks=1, in_blk=1024, out_blk=4096, bias=True, dtype="bf16"),
        # a ragged batch through odd blocks in single precision
        dict(name="backward_odd", op="backward", rows=301, nblocks=5, in_blk=77, out_blk=130, bias=True, dtype="f32"),
    ]


def draw(rng):
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    op = rng.choice(("quantise", "linear", "weights", "monarch", "backward"))
    if op == "quantise":
        case = dict(op=op, weights=rng.random() < 0.5, rows=size(1, 16384), nblocks=size(1, 16), cols=size(8, 4096), dtype=dtype)
        while case["rows"] * case["nblocks"] * case["cols"] > 1 << 26:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    if op == "monarch":
        rows = size(1, 64)
        if rng.random() < 0.5:  # square blocks, as many as they are wide
            b = size(8, 64)
            return dict(op=op, rows=rows, nb1=b, in1=b, out1=b, nb2=b, in2=b, out2=b, out_transpose=1, dtype=dtype)
        nb, i, o = size(2, 8), size(32, 1024), size(32, 1024)
        return dict(op=op, rows=rows, nb1=nb, in1=i, out1=min(i, o), nb2=nb, in2=min(i, o), out2=o, out_transpose=0, dtype=dtype)
    most_rows, most_work = {"linear": (16384, 1 << 37), "weights": (2048, 1 << 34), "backward": (8192, 1 << 35)}[op]
    case = dict(op=op, rows=size(1, most_rows), nblocks=size(1, 16), in_blk=size(16, 4096), out_blk=size(16, 4096),
                bias=rng.random() < 0.5, dtype=dtype)
    while case["nblocks"] * case["in_blk"] * case["out_blk"] > 1 << 24:  # weights of one layer
        case["nblocks"] = max(1, case["nblocks"] // 2)
    wide = case["nblocks"] * max(case["in_blk"], case["out_blk"])
    while case["rows"] * wide > 1 << 26 or case["rows"] * case["nblocks"] * case["in_blk"] * case["out_blk"] > most_work:
        case["rows"] = max(1, case["rows"] // 2)
    return case


def _mx4_bytes(rows, nblocks, cols):
    return rows * nblocks * ((cols + 31) // 32) * 17  # 32 values of 4 bits and their scale


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "quantise":
        n = c["rows"] * c["nblocks"] * c["cols"]
        return {"bytes": 2 * n * es + _mx4_bytes(c["rows"], c["nblocks"], c["cols"]), "flops": 4 * n}
    if c["op"] == "monarch":
        factors = _mx4_bytes(c["out1"], c["nb1"], c["in1"]) + _mx4_bytes(c["out2"], c["nb2"], c["in2"])
        return {"bytes": factors + c["rows"] * (c["nb1"] * c["in1"] + c["nb2"] * c["out2"]) * es,
                "flops": 2 * c["rows"] * (c["nb1"] * c["in1"] * c["out1"] + c["nb2"] * c["in2"] * c["out2"])}
    rows, nb, i, o = c["rows"], c["nblocks"], c["in_blk"], c["out_blk"]
    wq, xq, b = _mx4_bytes(o, nb, i), _mx4_bytes(rows, nb, i), nb * o * es if c["bias"] else 0
    if c["op"] == "backward":
        return {"bytes": wq + xq + b + (rows * nb * (o + i) + nb * o * i) * es, "flops": 4 * rows * nb * i * o}
    return {"bytes": wq + b + rows * nb * (i + o) * es, "flops": 2 * rows * nb * i * o}


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    """The plain tensors of a case, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def activations(rows, n):
        # a few channels far larger than the rest, as in a transformer's hidden states, and padded rows of zeros
        x = normal(rows, n) * torch.where(torch.rand(n, generator=g, device="cuda") < 1 / 64, 12.0, 1.0)
        x[rows - rows // 16:] = 0
        return x.to(dtype)

    def weights(nb, out, inn):
        return ((torch.rand((nb, out, inn), generator=g, device="cuda") * 2 - 1) / inn ** 0.5).to(dtype)

    c = case
    if c["op"] == "quantise":
        if c["weights"]:
            return {"X": weights(c["nblocks"], c["rows"], c["cols"])}
        return {"X": activations(c["rows"], c["nblocks"] * c["cols"])}
    if c["op"] == "monarch":
        return {"X": activations(c["rows"], c["nb1"] * c["in1"]), "R": weights(c["nb1"], c["out1"], c["in1"]),
                "L": weights(c["nb2"], c["out2"], c["in2"])}
    t = {"X": activations(c["rows"], c["nblocks"] * c["in_blk"]), "W": weights(c["nblocks"], c["out_blk"], c["in_blk"])}
    n_out = c["nblocks"] * c["out_blk"]
    if c["op"] == "backward":
        t["dY"] = normal(c["rows"], n_out).to(dtype)
    elif c["bias"]:
        t["bias"] = normal(n_out).to(dtype)
    return t


def prepare(case, seed):
    """What a program holds before the call: weights, and a backward's saved activations, stay in MX4
    (the framework's handle, or plain codes and scales)."""
    t = _inputs(case, seed)
    kept = {"linear": ("W",), "weights": ("W",), "monarch": ("R", "L"), "backward": ("X", "W")}.get(case["op"], ())
    if own:
        import block_diagonal_linear_b200 as bdl
        for k in kept:
            t[k] = bdl.mx4_quantise(t[k], nblocks=case["nblocks"]) if k == "X" else bdl.mx4_quantise(t[k])
    else:
        for k in kept:
            x = t[k].view(case["rows"], case["nblocks"], case["in_blk"]) if k == "X" else t[k]
            t[k] = _pack(x)
    return dict(t, case=case)


# ---------------------------------------------------------------- plain form
def _blocks(x):
    """x in 32 bits, its last axis in blocks of 32 (zeros behind the end)."""
    n = x.shape[-1]
    return torch.nn.functional.pad(x.float(), (0, -n % 32)).view(*x.shape[:-1], -1, 32)


def _scaled(x):
    """(values of x on the E2M1 grid, exponent of each block's scale)."""
    v = _blocks(x)
    e = torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 3  # frexp's mantissa lies in [0.5, 1)
    e = torch.where((v != 0).any(-1, keepdim=True), e, -127).clamp(-127, 125)
    a = torch.ldexp(v.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v), e


def _rounded(x):
    """x rounded to MX4 along its last axis, as 32-bit values of the same shape."""
    q, e = _scaled(x)
    return torch.ldexp(q, e).flatten(-2)[..., :x.shape[-1]]


def _pack(x):
    """(codes, two in a byte; scale bytes; length of the last axis) of x in MX4."""
    q, e = _scaled(x)
    code = torch.bucketize(q.abs(), torch.tensor(GRID, device=x.device)) + 8 * torch.signbit(q)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8), x.shape[-1]


def _values(packed):
    """The 32-bit values that _pack's result stands for."""
    codes, scales, n = packed
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    return torch.ldexp(v.unflatten(-1, (-1, 32)), scales.int().unsqueeze(-1) - 127).flatten(-2)[..., :n]


def _product(x, w):
    """(rows, nb, in) and (nb, out, in) -> (rows, nb, out)."""
    return torch.matmul(x.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1)


def _plain(s):
    c = s["case"]
    dtype, rows = DTYPES[c["dtype"]], c["rows"]
    if c["op"] == "quantise":
        x = s["X"] if c["weights"] else s["X"].view(rows, c["nblocks"], c["cols"])
        return _rounded(x).to(dtype).view(s["X"].shape)
    if c["op"] == "monarch":
        u = _product(s["X"].view(rows, c["nb1"], c["in1"]).float(), _values(s["R"]))
        z = u.transpose(1, 2).reshape(rows, c["nb2"], c["in2"])
        v = _product(z, _values(s["L"]))
        return (v.transpose(1, 2) if c["out_transpose"] else v).reshape(rows, -1).to(dtype)
    nb = c["nblocks"]
    if c["op"] == "backward":
        dy = s["dY"].view(rows, nb, c["out_blk"]).float()
        dx = torch.matmul(dy.transpose(0, 1), _values(s["W"])).transpose(0, 1)
        dw = torch.matmul(dy.permute(1, 2, 0), _values(s["X"]).transpose(0, 1))
        out = {"dX": dx.reshape(rows, -1).to(dtype), "dW": dw.to(dtype)}
        if c["bias"]:
            out["dbias"] = s["dY"].float().sum(0).to(dtype)
        return out
    x = s["X"].view(rows, nb, c["in_blk"])
    y = _product(_rounded(x) if c["op"] == "linear" else x.float(), _values(s["W"])).reshape(rows, -1)
    return (y + s["bias"].float() if c["bias"] else y).to(dtype)


def run(state):
    if not own:
        return _plain(state)
    import block_diagonal_linear_b200 as bdl
    s, c = state, state["case"]
    if c["op"] == "quantise":
        q = bdl.mx4_quantise(s["X"]) if c["weights"] else bdl.mx4_quantise(s["X"], nblocks=c["nblocks"])
        return bdl.mx4_dequantise(q, c["dtype"])
    if c["op"] == "linear":
        return bdl.mx4_linear_fwd(bdl.mx4_quantise(s["X"], nblocks=c["nblocks"]), s["W"], bias=s.get("bias"), dtype=c["dtype"])
    if c["op"] == "weights":
        return bdl.mx4_linear_fwd(s["X"], s["W"], bias=s.get("bias"))
    if c["op"] == "monarch":
        return bdl.mx4_fwd(s["X"], s["R"], s["L"], c)
    dX, dW, dbias = bdl.mx4_linear_bwd(s["dY"], s["X"], s["W"], bias=c["bias"])
    return {"dX": dX, "dW": dW, "dbias": dbias} if c["bias"] else {"dX": dX, "dW": dW}


# ---------------------------------------------------------------- the definition in 64 bits
def _mx4_64(x):
    """x in MX4 along its last axis by search among the sixteen values, in 64 bits."""
    n = x.shape[-1]
    pad = torch.zeros(*x.shape[:-1], -n % 32, dtype=torch.float64, device=x.device)
    v = torch.cat((x.double(), pad), -1).unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    # powers of two up to `top`: the count says floor(log2(top)) exactly, without a logarithm
    powers = torch.pow(2.0, torch.arange(-149, 128, dtype=torch.float64, device=x.device))
    scale = torch.pow(2.0, (torch.bucketize(top, powers, right=True) - 150.0 - 2.0).clamp(-127, 125))
    a = v.abs() / scale
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    k = torch.where(low % 2 == 0, low, high)  # on a tie the two differ: the even code of them
    return (torch.sign(v) * grid[k] * scale).flatten(-2)[..., :n]


def exact(case, seed):
    c, t = case, _inputs(case, seed)
    rows = c["rows"]
    if c["op"] == "quantise":
        x = t["X"] if c["weights"] else t["X"].view(rows, c["nblocks"], c["cols"])
        return _mx4_64(x).view(t["X"].shape)
    if c["op"] == "monarch":
        u = torch.einsum("rki,kpi->rpk", t["X"].double().view(rows, c["nb1"], c["in1"]), _mx4_64(t["R"]))
        z = u.reshape(rows, c["nb2"], c["in2"])
        v = torch.einsum("rjq,joq->" + ("roj" if c["out_transpose"] else "rjo"), z, _mx4_64(t["L"]))
        return v.reshape(rows, -1)
    nb = c["nblocks"]
    w = _mx4_64(t["W"])
    x = t["X"].view(rows, nb, c["in_blk"])
    if c["op"] == "backward":
        dy = t["dY"].double().view(rows, nb, c["out_blk"])
        out = {"dX": torch.einsum("rko,koi->rki", dy, w).reshape(rows, -1), "dW": torch.einsum("rko,rki->koi", dy, _mx4_64(x))}
        if c["bias"]:
            out["dbias"] = dy.sum(0).flatten()
        return out
    y = torch.einsum("rki,koi->rko", _mx4_64(x) if c["op"] == "linear" else x.double(), w).reshape(rows, -1)
    return y + t["bias"].double() if c["bias"] else y
