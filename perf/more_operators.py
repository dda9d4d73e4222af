"""Normalised rows and activations kept in 8 bits for the backward pass, as cases that can
be timed and compared.

A training step keeps what its backward pass reads: the rows that a norm read, the
inputs of its linear layers.  Kept as e4m3 codes, with one power of two for each 32
columns of a row, they take half of BF16's memory.  The cases are the root-mean-square
norm (with the residual's addition, and with its result in those 8 bits), its
gradients from either form of its input, writing and reading the 8-bit form, and a
linear layer's weight gradient from it.  ``run`` computes a case in a plain form
(elementary torch operations, in 32 bits, rounded once at the end) or, where ``own``
is true, through the package's entry points; ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
BLOCK = 32        # columns that share a scale
LARGEST = 448.0   # of e4m3
LEAST = -110      # exponent of the smallest scale


def listed():
    return [
        # --- norm of x + residual: y, the sum and 1/rms of each row
        # one token of a decoding step: launch latency is all there is
        dict(name="rms 1 token", op="rms_norm", mode="forward", rows=1, cols=4096, dtype="bf16"),
        # a decoding batch whose normalised rows feed 8-bit products
        dict(name="rms 8-bit 128 tokens", op="rms_norm", mode="8bit", rows=128, cols=4096,
             dtype="bf16"),
        # the same for a long prompt
        dict(name="rms 8-bit 16384x4096", op="rms_norm", mode="8bit", rows=16384, cols=4096,
             dtype="bf16"),
        # one layer's norm in a training step, both directions, everything kept in BF16
        dict(name="rms train 8192x4096", op="rms_norm", mode="train", rows=8192, cols=4096,
             dtype="bf16"),
        # the same with the norm's result and its input kept in 8 bits
        dict(name="rms train 8-bit 8192x4096", op="rms_norm", mode="train8", rows=8192, cols=4096,
             dtype="bf16"),
        # odd width: rows at every alignment, a last block of one column
        dict(name="rms train ragged f32", op="rms_norm", mode="train", rows=1000, cols=1025,
             dtype="f32"),
        # --- activations to 8 bits and back
        # a large batch's inputs of a linear layer
        dict(name="keep 16384x4096", op="keep", rows=16384, cols=4096, dtype="bf16"),
        # odd sizes in 32 bits
        dict(name="keep ragged f32", op="keep", rows=4095, cols=777, dtype="f32"),
        # --- weight gradient dy^T x of a linear layer whose x was kept in 8 bits
        # a small layer, few tokens
        dict(name="weight small", op="weight_grad", tokens=300, out=512, width=256, dtype="bf16"),
        # an ordinary layer and batch
        dict(name="weight 4096", op="weight_grad", tokens=4096, out=4096, width=4096, dtype="bf16"),
        # a large batch on a wide layer
        dict(name="weight 16384 wide", op="weight_grad", tokens=16384, out=11008, width=4096,
             dtype="bf16"),
        # odd sizes everywhere, gradients in 32 bits
        dict(name="weight ragged f32", op="weight_grad", tokens=1000, out=1025, width=777,
             dtype="f32"),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number of [lo, hi], its logarithm uniform, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, max(step, v // step * step)))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm", "keep", "weight_grad", "weight_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = rng.choice([1, 8, 32, 64])
    if op == "weight_grad":
        most = 16384 * 11008 * 4096 if dtype == "bf16" else 2 ** 37
        while True:
            c = dict(op=op, tokens=_spread(rng, 1, 16384), out=_spread(rng, 64, 11008, step),
                     width=_spread(rng, 64, 11008, step), dtype=dtype)
            if c["tokens"] * c["out"] * c["width"] <= most:
                return c
    mode = {} if op == "keep" else {"mode": rng.choice(["forward", "8bit", "train", "train8"])}
    while True:
        c = dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 64, 8192, step),
                 dtype=dtype, **mode)
        if c["rows"] * c["cols"] * (2 if dtype == "f32" else 1) <= 2 ** 26:
            return c


# ------------------------------------------------------------- the 8-bit form

def _power(e):
    """2^e in 32 bits, from whole exponents between -126 and 127."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x):
    """Codes (e4m3) and exponents of the scales of x's rows, in blocks of BLOCK columns.  The
    scale is the smallest power of two, 2^LEAST at least, that brings the block's largest
    finite value to LARGEST or below; infinities and NaN become NaN."""
    r, c = x.shape
    nb = -(-c // BLOCK)
    b = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - c)).view(r, nb, BLOCK)
    size = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).abs().amax(2)
    m, e = torch.frexp(size)           # size = m 2^e with m in [0.5, 1); LARGEST = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=LEAST)
    codes = (b * _power(-e)[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(r, nb * BLOCK)[:, :c], e


def _decode(codes, e):
    each = _power(e).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.float() * each


# -------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std).add_(mean)

    def activations(r, c):
        """Rows in which one column in a hundred is far larger than the others."""
        x = normal(r, c)
        x *= 1 + 15 * (torch.rand(c, generator=gen, device=dev) < 0.01).float()
        return x

    s = {"case": case}
    if case["op"] == "rms_norm":
        r, c = case["rows"], case["cols"]
        s["x"], s["residual"] = normal(r, c, std=0.5).to(dt), activations(r, c).to(dt)
        s["weight"] = normal(c, std=0.2, mean=1.0).to(dt)
        if case["mode"].startswith("train"):
            s["dy"], s["dtotal"] = normal(r, c, std=0.01).to(dt), normal(r, c, std=0.01).to(dt)
    elif case["op"] == "keep":
        s["x"] = activations(case["rows"], case["cols"]).to(dt)
    else:
        n, o, w = case["tokens"], case["out"], case["width"]
        s["dy"] = normal(n, o, std=0.01).to(dt)
        codes, e = _encode(activations(n, w))
        # rows on 16-byte boundaries, as the package lays the codes out
        q = torch.zeros(n, -(-w // 16) * 16, dtype=torch.uint8, device=dev)
        q[:, :w] = codes.contiguous().view(torch.uint8)
        s["codes"] = q.view(torch.float8_e4m3fn)[:, :w]
        s["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import dense_fp32_gemm_07_gb300 as b2g

    case = s["case"]
    if case["op"] == "rms_norm":
        args = dict(residual=s["residual"], eps=EPS)
        mode = case["mode"]
        if mode in ("forward", "train"):
            y, total, rstd = b2g.rms_norm(s["x"], s["weight"], **args)
            out, kept = {"y": y}, total
        else:
            train = mode == "train8"
            y, total, rstd, y8, kept = b2g.rms_norm_8bit(s["x"], s["weight"], with_y=train,
                                                         keep_total=train, **args)
            out = {"y": y} if train else {}
            out["y8"] = b2g.dequantize_8bit(*y8, torch.bfloat16)
        out["total"], out["rstd"] = total, rstd
        if mode.startswith("train"):
            out["dx"], out["dweight"] = b2g.rms_norm_backward(s["dy"], kept, s["weight"], rstd,
                                                              dtotal=s["dtotal"])
        return out
    if case["op"] == "keep":
        codes, scales = b2g.quantize_8bit(s["x"])
        return {"values": b2g.dequantize_8bit(codes, scales, s["x"].dtype)}
    return {"dw": b2g.linear_weight_grad_8bit(s["dy"], s["codes"], s["scales"])}


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "rms_norm":
        mode, w = case["mode"], s["weight"].float()
        total = (s["x"].float() + s["residual"].float()).to(dt)
        t = total.float()
        rstd = torch.rsqrt((t * t).mean(1) + EPS)
        y = t * rstd[:, None] * w
        out = {"total": total, "rstd": rstd}
        if mode != "8bit":
            out["y"] = y.to(dt)
        if mode.endswith("8") or mode == "8bit":
            out["y8"] = _decode(*_encode(y)).to(torch.bfloat16)
        if mode.startswith("train"):
            if mode == "train8":
                t = _decode(*_encode(t))
            dy = s["dy"].float()
            g, xhat = dy * w, t * rstd[:, None]
            dx = (g - xhat * (g * xhat).mean(1)[:, None]) * rstd[:, None] + s["dtotal"].float()
            out["dx"], out["dweight"] = dx.to(dt), (dy * xhat).sum(0).to(dt)
        return out
    if case["op"] == "keep":
        return {"values": _decode(*_encode(s["x"])).to(dt)}
    x = _decode(s["codes"], s["scales"].view(torch.uint8).int() - 127)
    return {"dw": (s["dy"].float().t() @ x).to(dt)}


# ------------------------------------------------------- the same in 64 bits

def _rounded64(x):
    """The values that x's 8-bit form stands for: each block's values to the nearest multiple
    (ties to the even one) of an eighth of their power of two, times the scale, or of the
    smallest code 2^-9 of it."""
    r, c = x.shape
    nb = -(-c // BLOCK)
    b = torch.zeros(r, nb * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :c] = x
    b = b.view(r, nb, BLOCK)
    size = b.abs().amax(2, keepdim=True).clamp(min=2.0 ** (LEAST - 1))
    scale = torch.exp2(torch.ceil(torch.log2(size / LARGEST)).clamp(min=LEAST))
    v = b / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * scale).view(r, nb * BLOCK)[:, :c]


def exact(case, seed):
    if case["op"] == "weight_grad" and 2 * case["tokens"] * case["out"] * case["width"] > 8e12:
        return None  # a 64-bit product would take too long
    s = prepare(case, seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "keep":
        return {"values": _rounded64(s["x"].double())}
    if case["op"] == "weight_grad":
        each = s["scales"].view(torch.uint8).double().sub(127).exp2()
        x = s["codes"].double() * each.repeat_interleave(BLOCK, 1)[:, :case["width"]]
        return {"dw": torch.einsum("to,tw->ow", s["dy"].double(), x)}
    mode = case["mode"]
    total = s["x"].double() + s["residual"].double()
    t = total.to(dt).double().requires_grad_()        # the norm is that of the stored sum
    w = s["weight"].double().requires_grad_()
    rstd = 1 / torch.sqrt(t.square().mean(1, keepdim=True) + EPS)
    y = t * rstd * w
    out = {"total": total, "rstd": rstd.detach()[:, 0]}
    if mode != "8bit":
        out["y"] = y.detach()
    if mode in ("8bit", "train8"):
        out["y8"] = _rounded64(y.detach())
    if mode == "train":
        y.backward(s["dy"].double())
        out["dx"], out["dweight"] = t.grad + s["dtotal"].double(), w.grad
    elif mode == "train8":   # the gradient's formula at the kept rows, with the forward's 1/rms
        n = _rounded64(t.detach()) * rstd.detach()
        g = s["dy"].double() * w.detach()
        along = (g * n).sum(1, keepdim=True) / case["cols"]
        out["dx"] = rstd.detach() * (g - along * n) + s["dtotal"].double()
        out["dweight"] = torch.einsum("rc,rc->c", s["dy"].double(), n)
    return out


# ------------------------------------- what a pass reads, writes and computes

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "weight_grad":
        n, o, w = case["tokens"], case["out"], case["width"]
        return {"bytes": n * o * es + n * w + n * -(-w // BLOCK) + o * w * es,
                "flops": 2 * n * o * w}
    n, kept = case["rows"] * case["cols"], case["rows"] * (case["cols"] + -(-case["cols"] // BLOCK))
    if case["op"] == "keep":                      # x, codes; codes, values
        return {"bytes": 2 * n * es + 2 * kept, "flops": 4 * n}
    mode, c = case["mode"], case["cols"]
    b, f = 3 * n * es + c * es + 4 * case["rows"], 5 * n   # x, residual, total; weight; rstd
    if mode != "8bit":
        b += n * es                               # y
    if mode in ("8bit", "train8"):                # codes written, read back as BF16
        b, f = b + 2 * kept + 2 * n, f + 4 * n
    if mode.startswith("train"):                  # dy, dtotal, dx; dweight; the kept rows
        b, f = b + 3 * n * es + c * es, f + 10 * n
        b += n * es if mode == "train" else 2 * kept
    return {"bytes": b, "flops": f}
