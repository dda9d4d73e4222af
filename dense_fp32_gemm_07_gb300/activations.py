"""Root-mean-square norm and activations kept in 8 bits for the backward pass
(include/b2g_train.h), next to the training-step operators of train.py and with their
rules: float32 or bfloat16 CUDA matrices with unit column stride, the current stream or
``stream``, TypeError or ValueError for wrong arguments, ``B2GError`` for library codes.

The 8-bit form of a rows x cols matrix is a pair of tensors:

    codes   torch.float8_e4m3fn, rows x cols (rows on 16-byte boundaries as made here)
    scales  torch.float8_e8m0fnu, rows x ceil(cols / 32): a power of two for each 32
            columns of a row

and stands for codes * scales.  The scale is the smallest power of two, 2^-110 at least,
that brings the block's largest finite value to 448 or below, so a value is rounded once,
by at most 2^-4 of itself or 2^-10 of the scale; infinities and NaN are kept as NaN.

Codes and scales made by a call with plain arguments share one storage, those of other calls
have one each: nothing should resize, free or move one of a pair by its storage, and saving
or keeping either keeps both.
"""
from __future__ import annotations

from . import B2G_ERR_INVALID_DIM, B2GError
from . import train as _train
from .train import _CODES, _apart, _matrix, _on, _plain, _result, _setup, _size, _vector

BLOCK = 32  # columns that share a scale


def _torch():
    return _train._torch


def _fast():
    return _train._fast or _setup()


def _codes(codes, scales, name):
    """(rows, columns, leading dimensions of the codes and of the scales, device number)."""
    if _train._torch is None:
        _setup()
    t = _torch()
    for x, dt, what in ((codes, t.float8_e4m3fn, "codes"), (scales, t.float8_e8m0fnu, "scales")):
        if not isinstance(x, t.Tensor) or x.dtype is not dt:
            raise TypeError(f"{name}: the {what} must be a {dt} tensor")
        if x.get_device() < 0:
            raise TypeError(f"{name}: the {what} must be on a CUDA device")
        if x.dim() != 2:
            raise ValueError(f"{name}: the {what} must be 2-D")
    r, c = codes.shape
    if tuple(scales.shape) != (r, -(-c // BLOCK)):
        raise ValueError(f"{name}: scales must be {r} x {-(-c // BLOCK)} for codes of {r} x {c}")
    dev = codes.get_device()
    if scales.get_device() != dev:
        raise ValueError(f"{name}: the scales must be on cuda:{dev}")
    lds = []
    for x, what in ((codes, "codes"), (scales, "scales")):
        n = x.shape[1]
        s0, s1 = x.stride()
        if n > 1 and s1 != 1:
            raise ValueError(f"{name}: the {what} must have unit column stride (row-major rows)")
        if r > 1 and s0 < n:
            raise ValueError(f"{name}: the {what} must not have overlapping rows")
        lds.append(s0 if r > 1 else max(1, n))
    return r, c, lds[0], lds[1], dev


def _length(*lengths):
    """Refuses lengths that the library's calls cannot take, before they are cut to 32 bits."""
    if max(lengths) > 0x7fffffff:
        raise B2GError(B2G_ERR_INVALID_DIM)


def _pair(x, name):
    if not isinstance(x, (tuple, list)) or len(x) != 2:
        raise TypeError(f"{name} must be a matrix or a pair of codes and scales")
    return x


def _new_codes(on, r, c, device):
    """Codes (rows on 16-byte boundaries), scales, and their leading dimensions."""
    t = _torch()
    ld, nb = -(-c // 16) * 16, -(-c // BLOCK)
    codes = on.empty((r, ld), t.float8_e4m3fn, device)[:, :c]
    return codes, on.empty((r, nb), t.float8_e8m0fnu, device), ld or 1, nb or 1


# -------------------------------------------------------------------- 8 bits

def quantize_8bit(x, stream=None):
    """(codes, scales) of a matrix: its 8-bit form."""
    if stream is None:
        got = _fast().quantize_8bit(x)
        if got is not None:
            return _plain(got)
    r, c, ldx = _matrix(x, "x")
    _length(c)
    dev = x.get_device()
    on = _on(stream, dev)
    codes, scales, ldq, lds = _new_codes(on, r, c, x.device)
    rc = _train._lib.b2g_quantize8(_CODES[x.dtype], r, c, x.data_ptr(), ldx, codes.data_ptr(), ldq,
                                   scales.data_ptr(), lds, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(x)
    return codes, scales


def dequantize_8bit(codes, scales, dtype=None, out=None, stream=None):
    """The matrix that an 8-bit form stands for, as `dtype` (torch.bfloat16 unless `out`,
    which takes the result, has another type)."""
    if out is None and stream is None:
        got = _fast().dequantize_8bit(codes, scales, dtype)
        if got is not None:
            return _plain(got)
    r, c, ldq, lds, dev = _codes(codes, scales, "dequantize_8bit")
    _length(c)
    t = _torch()
    if dtype is None:
        dtype = t.bfloat16 if out is None else out.dtype
    if dtype not in _CODES:
        raise TypeError("dtype must be torch.float32 or torch.bfloat16")
    on = _on(stream, dev)
    if out is None:
        out, ldy = on.empty((r, c), dtype, codes.device), c or 1
    else:
        ldy = _result(out, "out", (r, c), dtype, dev)
        _apart(out, ("codes", codes), ("scales", scales))
    rc = _train._lib.b2g_dequantize8(_CODES[dtype], r, c, codes.data_ptr(), ldq, scales.data_ptr(),
                                     lds, out.data_ptr(), ldy, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(codes, scales, out)
    return out


# ------------------------------------------------------------------ RMS norm

def rms_norm(x, weight=None, residual=None, eps: float = 1e-5, out=None, stream=None):
    """(y, total, rstd): total = x + residual, rounded to the type (x itself without a
    residual), and its rows divided by their root mean square, times `weight`.

    weight is a vector of cols elements of x's type (None: ones); rstd, 1 / sqrt(mean
    of total^2 + eps), a float32 vector for the backward pass.  `out` takes y and may be
    the residual itself or, where there is one, x (without one total is x)."""
    if out is None and stream is None:
        got = _fast().rms_norm(x, weight, residual, eps)
        if got is not None:
            return _plain(got)
    y, total, rstd, _, _ = _rms(x, weight, residual, eps, True, False, False, out, stream)
    return y, total, rstd


def rms_norm_8bit(x, weight=None, residual=None, eps: float = 1e-5, with_y: bool = False,
                  keep_total: bool = False, stream=None):
    """(y, total, rstd, y8, total8): `rms_norm` whose result leaves in 8 bits, y8 = (codes,
    scales), rounded once from FP32.

    y is None unless `with_y` asks for it in x's type too.  With `keep_total`, total8 is the
    8-bit form of total, for `rms_norm_backward`; otherwise None."""
    if stream is None:
        got = _fast().rms_norm_8bit(x, weight, residual, eps, with_y, keep_total)
        if got is not None:
            return _plain(got)
    return _rms(x, weight, residual, eps, with_y, True, keep_total, None, stream)


def _rms(x, weight, residual, eps, with_y, with_y8, with_t8, out, stream):
    r, c, ldx = _matrix(x, "x")
    dt, device, dev = x.dtype, x.device, x.get_device()
    _length(c)
    pr, ldr = None, 0
    if residual is not None:
        rr, cr, ldr = _matrix(residual, "residual", dt, dev)
        if (rr, cr) != (r, c):
            raise ValueError("residual must have x's shape")
        pr = residual.data_ptr()
    pw = _vector(weight, "weight", c, dt, dev)
    on = _on(stream, dev)
    y, ldy = None, 0
    if out is not None:
        y, ldy = out, _result(out, "out", (r, c), dt, dev)
        for name, t, ld in (("x", x, ldx), ("residual", residual, ldr)):
            if t is not None and (out.data_ptr() != t.data_ptr() or ldy != ld):
                _apart(out, (name, t))
        _apart(out, ("weight", weight))
        if residual is None and out.data_ptr() == x.data_ptr() and x.numel():
            # total would be x, which y overwrites
            raise ValueError("out may be x only with a residual")
    elif with_y:
        y, ldy = on.empty((r, c), dt, device), c or 1
    total = x if residual is None else on.empty((r, c), dt, device)
    rstd = on.empty((r,), _torch().float32, device)
    if c == 0:  # nothing is launched: rows of nothing have no mean
        on.fill(rstd, float("nan"))
    eight, pairs = [], []  # the arguments of the two 8-bit results, and the results
    for want in (with_y8, with_t8):
        if want:
            codes, scales, ldq, lds = _new_codes(on, r, c, device)
            eight += [codes.data_ptr(), ldq, scales.data_ptr(), lds]
            pairs.append((codes, scales))
        else:
            eight += [None, 0, None, 0]
            pairs.append(None)
    rc = _train._lib.b2g_rmsnorm(
        _CODES[dt], r, c, x.data_ptr(), ldx, pr, ldr, pw, eps,
        None if residual is None else total.data_ptr(), c or 1,
        None if y is None else y.data_ptr(), ldy, *eight, rstd.data_ptr(), on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(x, weight, residual, out)
    return y, total, rstd, pairs[0], pairs[1]


def rms_norm_backward(dy, total, weight, rstd, dtotal=None, out=None, stream=None):
    """(dx, dweight) of `rms_norm` for the gradient dy of y.

    total is the forward call's, or its 8-bit form as a pair (codes, scales); weight and
    rstd as there.  dtotal, the gradient that reaches total past the norm, is added to dx,
    which is the gradient of x and of the residual alike.  dweight is None when weight is.
    `out` takes dx and may be dy or dtotal itself."""
    if out is None and stream is None:
        got = _fast().rms_norm_backward(dy, total, weight, rstd, dtotal)
        if got is not None:
            return _plain(got)
    r, c, lddy = _matrix(dy, "dy")
    _length(c)
    dt, device, dev = dy.dtype, dy.device, dy.get_device()
    if isinstance(total, _torch().Tensor):
        rt, ct, ldt = _matrix(total, "total", dt, dev)
        kept, ps, lds = (total,), None, 0
    else:
        kept = codes, scales = _pair(total, "total")
        rt, ct, ldt, lds, dk = _codes(codes, scales, "total")
        if dk != dev:
            raise ValueError(f"total must be on cuda:{dev}")
        ps = scales.data_ptr()
    if (rt, ct) != (r, c):
        raise ValueError("total must have dy's shape")
    pw = _vector(weight, "weight", c, dt, dev)
    pr = _vector(rstd, "rstd", r, _torch().float32, dev)
    pd, lddt = None, 0
    if dtotal is not None:
        rd, cd, lddt = _matrix(dtotal, "dtotal", dt, dev)
        if (rd, cd) != (r, c):
            raise ValueError("dtotal must have dy's shape")
        pd = dtotal.data_ptr()
    on = _on(stream, dev)
    if out is None:
        out, lddx = on.empty((r, c), dt, device), c or 1
    else:
        lddx = _result(out, "out", (r, c), dt, dev)
        _apart(out, *(("total", t) for t in kept), ("weight", weight), ("rstd", rstd))
        for name, t, ld in (("dy", dy, lddy), ("dtotal", dtotal, lddt)):
            if t is not None and (out.data_ptr() != t.data_ptr() or lddx != ld):
                _apart(out, (name, t))
    dw = None if weight is None else on.empty((c,), dt, device)
    code = _CODES[dt]
    n = 0 if dw is None else _size(_train._lib.b2g_rmsnorm_backward_workspace_size, code, r, c)
    ws = on.empty((n,), _torch().uint8, device)
    rc = _train._lib.b2g_rmsnorm_backward(
        code, r, c, dy.data_ptr(), lddy, kept[0].data_ptr(), ldt, ps, lds, pw, pr, pd, lddt,
        out.data_ptr(), lddx, None if dw is None else dw.data_ptr(), ws.data_ptr(), n, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(dy, *kept, weight, rstd, dtotal, out)
    return out, dw


# ------------------------------------------------------- linear weight gradient

def linear_weight_grad_8bit(dy, codes, scales, dw=None, accumulate: bool = False, stream=None):
    """dy^T x: the weight gradient (outputs x inputs) of a linear layer y = x w^T whose
    input was kept in 8 bits as (codes, scales), tokens x inputs.  dy is tokens x outputs.

    `dw` takes the result; with `accumulate` it is added to the values there.  x's values
    are exact in the products (with scales of 2^-110 or more, as made here), which add up in
    float32; with float32 dy all its 24 bits take part, of values below 2^-110 what is left of
    them above 2^-134 (dy must be finite)."""
    if stream is None:
        got = _fast().linear_weight_grad_8bit(dy, codes, scales, dw, accumulate)
        if got is not None:
            return _plain(got)
    n, o, lddy = _matrix(dy, "dy")
    dt, device, dev = dy.dtype, dy.device, dy.get_device()
    nx, w, ldq, lds, dk = _codes(codes, scales, "x")
    if dk != dev:
        raise ValueError(f"codes must be on cuda:{dev}")
    if nx != n:
        raise ValueError(f"dy and codes must have the same number of rows: {n} and {nx}")
    _length(n, o, w)
    on = _on(stream, dev)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw, lddw = on.empty((o, w), dt, device), w or 1
    else:
        lddw = _result(dw, "dw", (o, w), dt, dev)
        _apart(dw, ("dy", dy), ("codes", codes), ("scales", scales))
    code, pdy = _CODES[dt], dy.data_ptr()
    nb = _size(_train._lib.b2g_linear_dweight8_workspace_size_ex, code, n, o, w, pdy, lddy,
               codes.data_ptr(), ldq)
    ws = on.empty((nb,), _torch().uint8, device)
    rc = _train._lib.b2g_linear_dweight8(code, n, o, w, pdy, lddy, codes.data_ptr(), ldq,
                                         scales.data_ptr(), lds, 1 if accumulate else 0,
                                         dw.data_ptr(), lddw, ws.data_ptr(), nb, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(dy, codes, scales, dw)
    return dw
