"""Training-step operators beside the SGEMM (include/b2g_train.h): layer norm,
embedding, softmax cross entropy of a linear layer, clipping by the gradient
norm.

Tensor-level calls on float32 or bfloat16 CUDA tensors.  Every step runs in the
CUDA library; torch supplies device memory (results and workspaces, from its
caching allocator) and the current stream.  A call given another ``stream``
runs there: the caller orders its inputs on that stream, and the results belong
to it.  Matrices are 2-D with unit column stride; their row stride is the
leading dimension.  Argument errors raise TypeError or ValueError, library error
codes ``B2GError``; ids and targets out of range are reported by ``b2g_status``
(``B2G_ERR_INDEX``), since finding them would need a synchronisation.

Calls with plain arguments (contiguous operands, results allocated by the call,
the current stream) go straight through the native binding
(csrc/train_binding.cpp); the checks here serve all others and name what is wrong.
"""
from __future__ import annotations

import bisect
import ctypes
import functools
from typing import Optional

from . import B2GError, _load, _stream_handle, _t

B2G_F32 = 0
B2G_BF16 = 1

B2G_ERR_INVALID_TYPE = -12
B2G_ERR_WORKSPACE = -13
B2G_ERR_INDEX = -14

# every symbol include/b2g_train.h declares
TRAIN_EXPORTS = (
    "b2g_layernorm", "b2g_layernorm_backward", "b2g_layernorm_backward_workspace_size",
    "b2g_embedding", "b2g_embedding_backward", "b2g_embedding_backward_workspace_size",
    "b2g_linear_xent", "b2g_linear_xent_backward", "b2g_linear_xent_workspace_size",
    "b2g_grad_norm", "b2g_clip_grad_norm", "b2g_grad_norm_workspace_size",
)

_lib = None


def train_library():
    """The loaded library with the argument types of these entry points set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _load()
    for name in TRAIN_EXPORTS:
        if not hasattr(lib, name):
            raise RuntimeError(f"the library does not export {name}; build it again")
    i, f, vp, ll, sz = (ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong,
                        ctypes.c_size_t)
    psz = ctypes.POINTER(ctypes.c_size_t)
    lib.b2g_layernorm.argtypes = [i, ll, i, vp, ll, vp, vp, f, vp, ll, vp, vp, vp]
    lib.b2g_layernorm_backward.argtypes = [i, ll, i, vp, ll, vp, ll, vp, vp, vp, vp, ll, vp, vp,
                                           vp, sz, vp]
    lib.b2g_layernorm_backward_workspace_size.argtypes = [i, ll, i, psz]
    lib.b2g_embedding.argtypes = [i, ll, i, i, vp, i, vp, ll, f, vp, ll, vp]
    lib.b2g_embedding_backward.argtypes = [i, ll, i, i, vp, i, vp, ll, f, ll, i, vp, ll, vp, sz,
                                           vp]
    lib.b2g_embedding_backward_workspace_size.argtypes = [i, ll, i, i, psz]
    lib.b2g_linear_xent.argtypes = [i, i, i, i, vp, ll, vp, ll, vp, i, ll, vp, vp, vp, sz, vp]
    lib.b2g_linear_xent_backward.argtypes = [i, i, i, i, vp, ll, vp, ll, vp, i, ll, vp, vp, vp,
                                             ll, i, vp, ll, vp, sz, vp]
    lib.b2g_linear_xent_workspace_size.argtypes = [i, i, i, i, vp, ll, vp, ll, i, psz]
    lib.b2g_grad_norm.argtypes = [i, i, vp, vp, vp, vp, sz, vp]
    lib.b2g_clip_grad_norm.argtypes = [i, i, vp, vp, f, vp, vp, vp, sz, vp]
    lib.b2g_grad_norm_workspace_size.argtypes = [i, i, vp, psz]
    _lib = lib
    return lib


_fast = None   # the native binding
_torch = None
_CODES = {}  # torch element type -> the library's code


def _setup():
    """torch, the table of element types, the library and its native binding, on
    first use.  There is no fallback where they have not been built."""
    global _torch, _fast
    train_library()
    _torch = _t()
    _CODES.update({_torch.float32: B2G_F32, _torch.bfloat16: B2G_BF16})
    from . import _train_binding

    _fast = _train_binding
    return _fast


def _plain(got):
    """What the binding answered for plain arguments: a result or an error code."""
    if got.__class__ is int:
        raise B2GError(got)
    return got


# The checks below run in every call; each looks at as few attributes as it can
# (a tensor's cost about 0.1 us each), and says what is wrong only once something is.

def _matrix(t, name, dt=None, dev=None):
    """(rows, columns, leading dimension) of a row-major CUDA matrix, of element
    type dt on device number dev where those are given."""
    if _torch is None:
        _setup()
    if not isinstance(t, _torch.Tensor) or t.dtype not in _CODES:
        raise TypeError(f"{name} must be a torch.float32 or torch.bfloat16 tensor")
    d = t.get_device()
    if d < 0:
        raise TypeError(f"{name} must be on a CUDA device")
    if dt is not None and t.dtype is not dt:
        raise TypeError(f"{name} must have the type {dt}")
    if dev is not None and d != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = shape
    if t.is_contiguous():
        return r, c, (c or 1)
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    if r > 1 and s0 < c:
        raise ValueError(f"{name} must not have overlapping rows")
    return r, c, (s0 if r > 1 else max(1, c))


def _vector(t, name, n, dt, dev):
    """The pointer of a contiguous vector of n elements of type dt; None stays None."""
    if t is None:
        return None
    if not isinstance(t, _torch.Tensor) or t.dtype is not dt:
        raise TypeError(f"{name} must be a {dt} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    return t.data_ptr()


def _indices(t, name, dev):
    """(pointer, count, bytes each) of a contiguous vector of row numbers."""
    size = None
    if isinstance(t, _torch.Tensor):
        size = 8 if t.dtype is _torch.int64 else 4 if t.dtype is _torch.int32 else None
    if size is None:
        raise TypeError(f"{name} must be a torch.int64 or torch.int32 tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector")
    return t.data_ptr(), t.shape[0], size


def _result(t, name, shape, dt, dev):
    """The leading dimension of a given result matrix."""
    r, c, ld = _matrix(t, name, dt, dev)
    if (r, c) != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}")
    return ld


def _apart(out, *inputs):
    """Raise when a given result shares memory with an input it must not overlap."""
    a0 = out.data_ptr()
    a1 = a0 + _span(out)
    for name, t in inputs:
        if t is None:
            continue
        b0 = t.data_ptr()
        if a0 < b0 + _span(t) and b0 < a1 and not _side_by_side(out, t):
            raise ValueError(f"the result must not overlap {name}")


def _side_by_side(a, b):
    """Whether two matrices are different columns of the same rows (one row stride, as
    in the halves of a wider matrix): their spans overlap, their elements do not."""
    if a.dim() != 2 or b.dim() != 2 or a.shape[0] < 2 or b.shape[0] < 2:
        return False
    row = a.stride(0) * a.element_size()
    if row != b.stride(0) * b.element_size():
        return False
    at = (b.data_ptr() - a.data_ptr()) % row  # where b's columns begin, from a's first one
    return at >= a.shape[1] * a.element_size() and at + b.shape[1] * b.element_size() <= row


def _span(t):
    """Bytes from a tensor's first element to the end of its last one."""
    if t.numel() == 0:
        return 0
    return (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


class _OnStream:
    """Where a call with a `stream` argument runs.  Its results and workspaces are
    allocated for that stream, and torch's allocator is told which tensors the
    stream works on, since memory that Python frees may otherwise be reused while
    it does."""

    def __init__(self, stream):
        self.handle = _stream_handle(stream)
        self.stream = (stream if isinstance(stream, _torch.cuda.Stream)
                       else _torch.cuda.ExternalStream(self.handle) if self.handle
                       else _torch.cuda.default_stream())

    def empty(self, shape, dtype, device):
        with _torch.cuda.stream(self.stream):
            return _torch.empty(shape, dtype=dtype, device=device)

    def fill(self, t, value):
        with _torch.cuda.stream(self.stream):
            t.fill_(value)

    def uses(self, *tensors):
        for t in tensors:
            if t is not None:
                t.record_stream(self.stream)


class _OnCurrent:
    """A call on the current stream of a device: torch allocates for that stream."""

    __slots__ = ("handle", "empty")

    def __init__(self, dev):
        self.handle = _torch._C._cuda_getCurrentRawStream(dev)
        self.empty = _empty

    def fill(self, t, value):
        t.fill_(value)

    def uses(self, *tensors):
        pass


def _empty(shape, dtype, device):
    return _torch.empty(shape, dtype=dtype, device=device)


def _on(stream, dev):
    """The stream a call on device number dev runs on; the library's calls run on
    the current device, which has to be that one."""
    if dev != _torch._C._cuda_getDevice():
        raise ValueError(f"cuda:{dev} must be the current device")
    return _OnCurrent(dev) if stream is None else _OnStream(stream)


def _size(query, *args):
    """The workspace size that a query names."""
    n = ctypes.c_size_t(0)
    rc = query(*args, ctypes.byref(n))
    if rc:
        raise B2GError(rc)
    return n.value


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """(y, mean, rstd): each row of x normalised, times `weight`, plus `bias`.

    x is rows x cols; weight and bias are vectors of cols elements of its type
    (None: ones, zeros).  mean and rstd are float32 vectors for the backward pass.
    `out` takes y and may be x itself."""
    if out is None and stream is None:
        got = (_fast or _setup()).layer_norm(x, weight, bias, eps)
        if got is not None:
            return _plain(got)
    r, c, ldx = _matrix(x, "x")
    dt, device, dev = x.dtype, x.device, x.get_device()
    pw, pb = _vector(weight, "weight", c, dt, dev), _vector(bias, "bias", c, dt, dev)
    on = _on(stream, dev)
    if out is None:
        out, ldy = on.empty((r, c), dt, device), c or 1
    else:
        ldy = _result(out, "out", (r, c), dt, dev)
        if out.data_ptr() != x.data_ptr() or ldx != ldy:
            _apart(out, ("x", x))
        _apart(out, ("weight", weight), ("bias", bias))
    mean = on.empty((r,), _torch.float32, device)
    rstd = on.empty((r,), _torch.float32, device)
    if c == 0:  # nothing is launched: rows of nothing have no mean
        on.fill(mean, float("nan"))
        on.fill(rstd, float("nan"))
    rc = _lib.b2g_layernorm(_CODES[dt], r, c, x.data_ptr(), ldx, pw, pb, eps, out.data_ptr(), ldy,
                            mean.data_ptr(), rstd.data_ptr(), on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(x, weight, bias, out)
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True, out=None, stream=None):
    """(dx, dweight, dbias) of `layer_norm` for the gradient dy of y.

    weight, mean and rstd as in the forward call; dweight is None when weight is
    None, dbias when `bias` is false.  `out` takes dx and may be dy itself."""
    if out is None and stream is None:
        got = (_fast or _setup()).layer_norm_backward(dy, x, weight, mean, rstd, bias)
        if got is not None:
            return _plain(got)
    r, c, ldx = _matrix(x, "x")
    dt, device, dev = x.dtype, x.device, x.get_device()
    rd, cd, lddy = _matrix(dy, "dy", dt, dev)
    if rd != r or cd != c:
        raise ValueError("dy must have x's shape")
    pw = _vector(weight, "weight", c, dt, dev)
    pm = _vector(mean, "mean", r, _torch.float32, dev)
    pr = _vector(rstd, "rstd", r, _torch.float32, dev)
    on = _on(stream, dev)
    if out is None:
        out, lddx = on.empty((r, c), dt, device), c or 1
    else:
        lddx = _result(out, "out", (r, c), dt, dev)
        _apart(out, ("x", x), ("weight", weight), ("mean", mean), ("rstd", rstd))
        if out.data_ptr() != dy.data_ptr() or lddx != lddy:
            _apart(out, ("dy", dy))
    dw = None if weight is None else on.empty((c,), dt, device)
    db = on.empty((c,), dt, device) if bias else None
    code = _CODES[dt]
    n = _size(_lib.b2g_layernorm_backward_workspace_size, code, r, c)
    ws = on.empty((n,), _torch.uint8, device)
    rc = _lib.b2g_layernorm_backward(
        code, r, c, dy.data_ptr(), lddy, x.data_ptr(), ldx, pw, pm, pr, out.data_ptr(), lddx,
        None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
        ws.data_ptr(), n, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(dy, x, weight, mean, rstd, out)
    return out, dw, db


# ------------------------------------------------------------------- embedding

def embedding(ids, table, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids], one row per id; an id out of range gives a row of NaN."""
    if out is None and stream is None:
        got = (_fast or _setup()).embedding(ids, table, scale)
        if got is not None:
            return _plain(got)
    v, d, ldt = _matrix(table, "table")
    dt, device, dev = table.dtype, table.device, table.get_device()
    pi, n, width = _indices(ids, "ids", dev)
    on = _on(stream, dev)
    if out is None:
        out, ldo = on.empty((n, d), dt, device), d or 1
    else:
        ldo = _result(out, "out", (n, d), dt, dev)
        _apart(out, ("table", table), ("ids", ids))
    rc = _lib.b2g_embedding(_CODES[dt], n, v, d, pi, width, table.data_ptr(), ldt, scale,
                            out.data_ptr(), ldo, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(ids, table, out)
    return out


def embedding_backward(ids, dout, num_rows: int, scale: float = 1.0, out=None,
                       accumulate: bool = False, padding_idx: Optional[int] = None, stream=None):
    """The gradient of a table of num_rows rows: row v is scale times the sum of
    the rows of dout whose id is v, except padding_idx.  With `accumulate` it is
    added to `out`'s values (only rows with a token are touched)."""
    if out is None and padding_idx is None and stream is None and not accumulate:
        got = (_fast or _setup()).embedding_backward(ids, dout, num_rows, scale)
        if got is not None:
            return _plain(got)
    n, d, ldd = _matrix(dout, "dout")
    dt, device, dev = dout.dtype, dout.device, dout.get_device()
    pi, ni, width = _indices(ids, "ids", dev)
    if ni != n:
        raise ValueError("ids and dout must have the same number of rows")
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    if padding_idx is not None and not 0 <= padding_idx < num_rows:
        raise ValueError("padding_idx must be a row of the table")
    on = _on(stream, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out, ldt = on.empty((num_rows, d), dt, device), d or 1
    else:
        ldt = _result(out, "out", (num_rows, d), dt, dev)
        _apart(out, ("dout", dout), ("ids", ids))
    code = _CODES[dt]
    nb = _size(_lib.b2g_embedding_backward_workspace_size, code, n, num_rows, d)
    ws = on.empty((nb,), _torch.uint8, device)
    rc = _lib.b2g_embedding_backward(code, n, num_rows, d, pi, width, dout.data_ptr(), ldd, scale,
                                     -1 if padding_idx is None else padding_idx,
                                     1 if accumulate else 0, out.data_ptr(), ldt, ws.data_ptr(),
                                     nb, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(ids, dout, out)
    return out


# --------------------------------------------------------------- cross entropy

def linear_cross_entropy(h, w, target, ignore_index: int = -100, stream=None):
    """(loss, lse) per row of the logits h @ w.T, which are never stored.

    h is tokens x width, w vocab x width, target a vector of class numbers.
    loss_i = lse_i - logit_{i, target_i}, 0 where target_i is ignore_index; lse is
    the log of the sum of the exponentials.  Both are float32 vectors."""
    if stream is None:
        got = (_fast or _setup()).linear_cross_entropy(h, w, target, ignore_index)
        if got is not None:
            return _plain(got)
    n, d, ldh = _matrix(h, "h")
    dt, device, dev = h.dtype, h.device, h.get_device()
    v, dw, ldw = _matrix(w, "w", dt, dev)
    pt, nt, width = _indices(target, "target", dev)
    if dw != d or nt != n:
        raise ValueError(f"shape mismatch: h {n}x{d}, w {v}x{dw}, target {nt}")
    on = _on(stream, dev)
    loss = on.empty((n,), _torch.float32, device)
    lse = on.empty((n,), _torch.float32, device)
    code, ph, pw = _CODES[dt], h.data_ptr(), w.data_ptr()
    nb = _size(_lib.b2g_linear_xent_workspace_size, code, n, v, d, ph, ldh, pw, ldw, 0)
    ws = on.empty((nb,), _torch.uint8, device)
    rc = _lib.b2g_linear_xent(code, n, v, d, ph, ldh, pw, ldw, pt, width, ignore_index,
                              loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(h, w, target)
    return loss, lse


def linear_cross_entropy_backward(h, w, target, lse, grad_loss, ignore_index: int = -100,
                                  dw=None, accumulate: bool = False, stream=None):
    """(dh, dw): gradients of (grad_loss * loss).sum() for `linear_cross_entropy`.

    lse is the forward call's; grad_loss a float32 vector, one weight per row
    (1 / n for a mean over n rows).  `dw` takes the head's gradient; with
    `accumulate` it is added to the values there."""
    if dw is None and stream is None and not accumulate:
        got = (_fast or _setup()).linear_cross_entropy_backward(h, w, target, lse, grad_loss,
                                                               ignore_index)
        if got is not None:
            return _plain(got)
    n, d, ldh = _matrix(h, "h")
    dt, device, dev = h.dtype, h.device, h.get_device()
    v, dv, ldw = _matrix(w, "w", dt, dev)
    pt, nt, width = _indices(target, "target", dev)
    if dv != d or nt != n:
        raise ValueError(f"shape mismatch: h {n}x{d}, w {v}x{dv}, target {nt}")
    pl = _vector(lse, "lse", n, _torch.float32, dev)
    pg = _vector(grad_loss, "grad_loss", n, _torch.float32, dev)
    on = _on(stream, dev)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw, lddw = on.empty((v, d), dt, device), d or 1
    else:
        lddw = _result(dw, "dw", (v, d), dt, dev)
        _apart(dw, ("h", h), ("w", w), ("target", target), ("lse", lse), ("grad_loss", grad_loss))
    dh = on.empty((n, d), dt, device)
    code, ph, pw = _CODES[dt], h.data_ptr(), w.data_ptr()
    nb = _size(_lib.b2g_linear_xent_workspace_size, code, n, v, d, ph, ldh, pw, ldw, 1)
    ws = on.empty((nb,), _torch.uint8, device)
    rc = _lib.b2g_linear_xent_backward(code, n, v, d, ph, ldh, pw, ldw, pt, width, ignore_index,
                                       pl, pg, dh.data_ptr(), d or 1, 1 if accumulate else 0,
                                       dw.data_ptr(), lddw, ws.data_ptr(), nb, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(h, w, target, lse, grad_loss, dw)
    return dh, dw


# ------------------------------------------------------------- gradient clipping

def _tensor_list(tensors, name, dt=None, dev=None):
    """(element type, device number, addresses, lengths) of a list of contiguous
    tensors of one type on one device."""
    if _torch is None:
        _setup()
    if not tensors:
        raise ValueError(f"{name} must hold at least one tensor")
    if dt is None:
        first = tensors[0]
        if not isinstance(first, _torch.Tensor) or first.dtype not in _CODES:
            raise TypeError(f"{name} must hold torch.float32 or torch.bfloat16 tensors")
        dt, dev = first.dtype, first.get_device()
        if dev < 0:
            raise TypeError(f"{name} must be on a CUDA device")
    for t in tensors:
        if not isinstance(t, _torch.Tensor) or t.dtype is not dt:
            raise TypeError(f"{name} must hold {dt} tensors only")
        if not t.is_contiguous() or t.get_device() != dev:
            raise ValueError(f"every tensor of {name} must be contiguous and on cuda:{dev}")
    return dt, dev, [t.data_ptr() for t in tensors], [t.numel() for t in tensors]


def grad_norm(grads, stream=None):
    """The 2-norm of all elements of the tensors in the list, a 0-d float32 tensor."""
    grads = list(grads)
    if stream is None:
        got = (_fast or _setup()).clip(grads)
        if got is not None:
            return _plain(got)
    return _norm(grads, None, None, stream)


def clip_grad_norm(grads, max_norm: float, out=None, stream=None):
    """Multiply every tensor of the list by min(1, max_norm / (norm + 1e-6)), with
    the 2-norm of all of them together, and return that norm (a 0-d float32
    tensor).  In place, or into the tensors of the list `out`.  No result may share
    memory with another one (so no tensor may be clipped in place twice), nor with a
    tensor of `grads` other than the one it replaces."""
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    grads = list(grads)
    outs = grads if out is None else list(out)
    if stream is None:
        got = (_fast or _setup()).clip(grads, outs, max_norm)
        if got is not None:
            return _plain(got)
    return _norm(grads, outs, max_norm, stream)


def _norm(grads, outs, max_norm, stream):
    dt, dev, ptrs, lens = _tensor_list(grads, "grads")
    n = len(ptrs)
    optrs = ptrs
    if outs is not None and outs is not grads:
        _, _, optrs, olens = _tensor_list(outs, "out", dt, dev)
        if olens != lens:
            raise ValueError("out must hold tensors of the lengths of grads")
    if outs is not None:
        _all_apart(ptrs, optrs, lens, grads[0].element_size())
    on = _on(stream, dev)
    device = grads[0].device
    norm = on.empty((), _torch.float32, device)
    code, table = _CODES[dt], _ADDRESSES(n)
    addresses, lengths = table(*ptrs), table(*lens)
    nb = _size(_lib.b2g_grad_norm_workspace_size, code, n, lengths)
    ws = on.empty((nb,), _torch.uint8, device)
    if outs is None:
        rc = _lib.b2g_grad_norm(code, n, addresses, lengths, norm.data_ptr(), ws.data_ptr(), nb,
                                on.handle)
    else:
        rc = _lib.b2g_clip_grad_norm(code, n, addresses, lengths, max_norm,
                                     addresses if optrs is ptrs else table(*optrs),
                                     norm.data_ptr(), ws.data_ptr(), nb, on.handle)
    if rc:
        raise B2GError(rc)
    on.uses(*grads, *(outs or ()))
    return norm


def _all_apart(ptrs, optrs, lens, bytes_each):
    """Raise when a result of a list shares memory with another one, or with an input
    other than the tensor it replaces."""
    def spans(at):
        return [(p, p + n * bytes_each, i) for i, (p, n) in enumerate(zip(at, lens)) if n]

    outs = sorted(spans(optrs))
    for (_, end, i), (start, _, j) in zip(outs, outs[1:]):
        if start < end:
            raise ValueError(f"the results of tensors {min(i, j)} and {max(i, j)} overlap")
    starts = [o[0] for o in outs]
    for start, end, i in spans(ptrs) if optrs is not ptrs else ():
        k = bisect.bisect_left(starts, end) - 1
        while k >= 0 and outs[k][1] > start:
            if outs[k][2] != i or outs[k][0] != start:
                raise ValueError(f"the result of tensor {outs[k][2]} must not overlap tensor {i}")
            k -= 1


@functools.lru_cache(maxsize=None)
def _ADDRESSES(n):
    """The ctypes array type of n 64-bit addresses or lengths."""
    return ctypes.c_longlong * n
