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
"""
from __future__ import annotations

import ctypes
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


_codes = None


def _dtype(t, name, like=None):
    """The library's code of a tensor's element type (`like`: the type it must have)."""
    global _codes
    torch = _t()
    if _codes is None:
        _codes = {torch.float32: B2G_F32, torch.bfloat16: B2G_BF16}
    if not isinstance(t, torch.Tensor) or t.dtype not in _codes:
        raise TypeError(f"{name} must be a torch.float32 or torch.bfloat16 tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    if like is not None and t.dtype is not like.dtype:
        raise TypeError(f"{name} must have the type {like.dtype}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    return _codes[t.dtype]


def _matrix(t, name, like=None):
    """(type code, rows, columns, leading dimension) of a row-major matrix."""
    code = _dtype(t, name, like)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = t.shape
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride (row-major rows)")
    if r > 1 and s0 < c:
        raise ValueError(f"{name} must not have overlapping rows")
    return code, r, c, (s0 if r > 1 else max(1, c))


def _vector(t, name, n, like):
    """The pointer of a vector of n elements of `like`'s type; None stays None."""
    if t is None:
        return None
    _dtype(t, name, like)
    if t.dim() != 1 or t.size(0) != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    return t.data_ptr()


def _floats(t, name, n, like):
    """The pointer of a contiguous float32 vector of n elements."""
    torch = _t()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a torch.float32 tensor")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if t.dim() != 1 or t.size(0) != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    return t.data_ptr()


def _indices(t, name, like):
    """(pointer, count, bytes each) of a contiguous vector of row numbers."""
    torch = _t()
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"{name} must be a torch.int64 or torch.int32 tensor")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if t.dim() != 1 or (t.size(0) > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector")
    return t.data_ptr(), t.size(0), t.element_size()


def _result(t, name, shape, like):
    """The leading dimension of a given result matrix."""
    _, r, c, ld = _matrix(t, name, like)
    if (r, c) != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}")
    return ld


def _apart(out, *inputs):
    """Raise when a given result shares memory with an input it must not overlap."""
    a0 = out.data_ptr()
    a1 = a0 + _span(out)
    for name, t in inputs:
        b0 = t.data_ptr()
        if a0 < b0 + _span(t) and b0 < a1:
            raise ValueError(f"the result must not overlap {name}")


def _span(t):
    """Bytes from a tensor's first element to the end of its last one."""
    if t.numel() == 0:
        return 0
    return (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


class _On:
    """The stream a call runs on.  Results and workspaces are allocated for it:
    with a `stream` given, torch's allocator is told so, since memory freed by
    Python may otherwise be reused while that stream still works on it."""

    def __init__(self, stream):
        self.handle = _stream_handle(stream)
        self.other = None
        if stream is not None:
            torch = _t()
            self.other = (stream if isinstance(stream, torch.cuda.Stream)
                          else torch.cuda.ExternalStream(self.handle) if self.handle
                          else torch.cuda.default_stream())

    def empty(self, shape, dtype, device):
        torch = _t()
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.other):
            return torch.empty(shape, dtype=dtype, device=device)

    def uses(self, *tensors):
        """Inputs of another stream's allocator stay reserved until this stream is done."""
        if self.other is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.other)


def _raise(rc):
    if rc:
        raise B2GError(rc)


def _workspace(on, device, query, *args):
    """(tensor to keep alive, pointer, bytes) of the size a query names."""
    n = ctypes.c_size_t(0)
    _raise(query(*args, ctypes.byref(n)))
    if n.value == 0:
        return None, None, 0
    ws = on.empty((n.value,), _t().uint8, device)
    return ws, ws.data_ptr(), n.value


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None):
    """(y, mean, rstd): each row of x normalised, times `weight`, plus `bias`.

    x is rows x cols; weight and bias are vectors of cols elements of its type
    (None: ones, zeros).  mean and rstd are float32 vectors for the backward pass.
    `out` takes y and may be x itself."""
    lib = train_library()
    torch = _t()
    code, r, c, ldx = _matrix(x, "x")
    pw, pb = _vector(weight, "weight", c, x), _vector(bias, "bias", c, x)
    on = _On(stream)
    if out is None:
        out, ldy = on.empty((r, c), x.dtype, x.device), max(1, c)
    else:
        ldy = _result(out, "out", (r, c), x)
        if out.data_ptr() != x.data_ptr() or ldx != ldy:
            _apart(out, ("x", x))
    mean = on.empty((r,), torch.float32, x.device)
    rstd = on.empty((r,), torch.float32, x.device)
    _raise(lib.b2g_layernorm(code, r, c, x.data_ptr(), ldx, pw, pb, float(eps), out.data_ptr(),
                             ldy, mean.data_ptr(), rstd.data_ptr(), on.handle))
    on.uses(x, weight, bias, out)
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, bias: bool = True, out=None, stream=None):
    """(dx, dweight, dbias) of `layer_norm` for the gradient dy of y.

    weight, mean and rstd as in the forward call; dweight is None when weight is
    None, dbias when `bias` is false.  `out` takes dx and may be dy itself."""
    lib = train_library()
    code, r, c, ldx = _matrix(x, "x")
    _, rd, cd, lddy = _matrix(dy, "dy", x)
    if (rd, cd) != (r, c):
        raise ValueError("dy must have x's shape")
    pw = _vector(weight, "weight", c, x)
    pm, pr = _floats(mean, "mean", r, x), _floats(rstd, "rstd", r, x)
    on = _On(stream)
    if out is None:
        out, lddx = on.empty((r, c), x.dtype, x.device), max(1, c)
    else:
        lddx = _result(out, "out", (r, c), x)
        _apart(out, ("x", x))
        if out.data_ptr() != dy.data_ptr() or lddx != lddy:
            _apart(out, ("dy", dy))
    dw = on.empty((c,), x.dtype, x.device) if weight is not None else None
    db = on.empty((c,), x.dtype, x.device) if bias else None
    ws, p, n = _workspace(on, x.device, lib.b2g_layernorm_backward_workspace_size, code, r, c)
    _raise(lib.b2g_layernorm_backward(
        code, r, c, dy.data_ptr(), lddy, x.data_ptr(), ldx, pw, pm, pr, out.data_ptr(), lddx,
        None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(), p, n,
        on.handle))
    on.uses(dy, x, weight, mean, rstd, out)
    return out, dw, db


# ------------------------------------------------------------------- embedding

def embedding(ids, table, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids], one row per id; an id out of range gives a row of NaN."""
    lib = train_library()
    code, v, d, ldt = _matrix(table, "table")
    pi, n, width = _indices(ids, "ids", table)
    on = _On(stream)
    if out is None:
        out, ldo = on.empty((n, d), table.dtype, table.device), max(1, d)
    else:
        ldo = _result(out, "out", (n, d), table)
        _apart(out, ("table", table), ("ids", ids))
    _raise(lib.b2g_embedding(code, n, v, d, pi, width, table.data_ptr(), ldt, float(scale),
                             out.data_ptr(), ldo, on.handle))
    on.uses(ids, table, out)
    return out


def embedding_backward(ids, dout, num_rows: int, scale: float = 1.0, out=None,
                       accumulate: bool = False, padding_idx: Optional[int] = None, stream=None):
    """The gradient of a table of num_rows rows: row v is scale times the sum of
    the rows of dout whose id is v, except padding_idx.  With `accumulate` it is
    added to `out`'s values (only rows with a token are touched)."""
    lib = train_library()
    code, n, d, ldd = _matrix(dout, "dout")
    pi, ni, width = _indices(ids, "ids", dout)
    if ni != n:
        raise ValueError("ids and dout must have the same number of rows")
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    if padding_idx is not None and not 0 <= padding_idx < num_rows:
        raise ValueError("padding_idx must be a row of the table")
    on = _On(stream)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out, ldt = on.empty((num_rows, d), dout.dtype, dout.device), max(1, d)
    else:
        ldt = _result(out, "out", (num_rows, d), dout)
        _apart(out, ("dout", dout), ("ids", ids))
    ws, p, nb = _workspace(on, dout.device, lib.b2g_embedding_backward_workspace_size, code, n,
                           num_rows, d)
    _raise(lib.b2g_embedding_backward(code, n, num_rows, d, pi, width, dout.data_ptr(), ldd,
                                      float(scale), -1 if padding_idx is None else padding_idx,
                                      int(accumulate), out.data_ptr(), ldt, p, nb, on.handle))
    on.uses(ids, dout, out)
    return out


# --------------------------------------------------------------- cross entropy

def linear_cross_entropy(h, w, target, ignore_index: int = -100, stream=None):
    """(loss, lse) per row of the logits h @ w.T, which are never stored.

    h is tokens x width, w vocab x width, target a vector of class numbers.
    loss_i = lse_i - logit_{i, target_i}, 0 where target_i is ignore_index; lse is
    the log of the sum of the exponentials.  Both are float32 vectors."""
    lib = train_library()
    torch = _t()
    code, n, d, ldh = _matrix(h, "h")
    _, v, dw, ldw = _matrix(w, "w", h)
    pt, nt, width = _indices(target, "target", h)
    if dw != d or nt != n:
        raise ValueError(f"shape mismatch: h {n}x{d}, w {v}x{dw}, target {nt}")
    on = _On(stream)
    loss = on.empty((n,), torch.float32, h.device)
    lse = on.empty((n,), torch.float32, h.device)
    ws, p, nb = _workspace(on, h.device, lib.b2g_linear_xent_workspace_size, code, n, v, d,
                           h.data_ptr(), ldh, w.data_ptr(), ldw, 0)
    _raise(lib.b2g_linear_xent(code, n, v, d, h.data_ptr(), ldh, w.data_ptr(), ldw, pt, width,
                               ignore_index, loss.data_ptr(), lse.data_ptr(), p, nb, on.handle))
    on.uses(h, w, target)
    return loss, lse


def linear_cross_entropy_backward(h, w, target, lse, grad_loss, ignore_index: int = -100,
                                  dw=None, accumulate: bool = False, stream=None):
    """(dh, dw): gradients of (grad_loss * loss).sum() for `linear_cross_entropy`.

    lse is the forward call's; grad_loss a float32 vector, one weight per row
    (1 / n for a mean over n rows).  `dw` takes the head's gradient; with
    `accumulate` it is added to the values there."""
    lib = train_library()
    code, n, d, ldh = _matrix(h, "h")
    _, v, dh_, ldw = _matrix(w, "w", h)
    pt, nt, width = _indices(target, "target", h)
    if dh_ != d or nt != n:
        raise ValueError(f"shape mismatch: h {n}x{d}, w {v}x{dh_}, target {nt}")
    pl, pg = _floats(lse, "lse", n, h), _floats(grad_loss, "grad_loss", n, h)
    on = _On(stream)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw, lddw = on.empty((v, d), h.dtype, h.device), max(1, d)
    else:
        lddw = _result(dw, "dw", (v, d), h)
        _apart(dw, ("h", h), ("w", w))
    dh = on.empty((n, d), h.dtype, h.device)
    ws, p, nb = _workspace(on, h.device, lib.b2g_linear_xent_workspace_size, code, n, v, d,
                           h.data_ptr(), ldh, w.data_ptr(), ldw, 1)
    _raise(lib.b2g_linear_xent_backward(
        code, n, v, d, h.data_ptr(), ldh, w.data_ptr(), ldw, pt, width, ignore_index, pl, pg,
        dh.data_ptr(), max(1, d), int(accumulate), dw.data_ptr(), lddw, p, nb, on.handle))
    on.uses(h, w, target, lse, grad_loss, dw)
    return dh, dw


# ------------------------------------------------------------- gradient clipping

def _tensor_list(tensors, name):
    """(type code, pointer array, length array, device) of a list of contiguous tensors."""
    torch = _t()
    if not tensors:
        raise ValueError(f"{name} must hold at least one tensor")
    first = tensors[0]
    code = _dtype(first, f"{name}[0]")
    dt, dev = first.dtype, first.device
    for i, t in enumerate(tensors):
        if t.dtype is not dt or t.device != dev:
            raise TypeError(f"{name}[{i}] must have the type and device of {name}[0]")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
    n = len(tensors)
    return (code, (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]),
            (ctypes.c_longlong * n)(*[t.numel() for t in tensors]), dev)


def grad_norm(grads, stream=None):
    """The 2-norm of all elements of the tensors in the list, a 0-d float32 tensor."""
    return _norm(list(grads), None, None, stream)


def clip_grad_norm(grads, max_norm: float, out=None, stream=None):
    """Multiply every tensor of the list by min(1, max_norm / (norm + 1e-6)), with
    the 2-norm of all of them together, and return that norm (a 0-d float32
    tensor).  In place, or into the tensors of the list `out`."""
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    grads = list(grads)
    outs = grads if out is None else list(out)
    return _norm(grads, outs, float(max_norm), stream)


def _norm(grads, outs, max_norm, stream):
    lib = train_library()
    torch = _t()
    code, ptrs, numels, dev = _tensor_list(grads, "grads")
    n = len(grads)
    on = _On(stream)
    norm = on.empty((), torch.float32, dev)
    ws, p, nb = _workspace(on, dev, lib.b2g_grad_norm_workspace_size, code, n, numels)
    if outs is None:
        _raise(lib.b2g_grad_norm(code, n, ptrs, numels, norm.data_ptr(), p, nb, on.handle))
        on.uses(*grads)
        return norm
    optrs = ptrs
    if outs is not grads:
        ocode, optrs, olens, odev = _tensor_list(outs, "out")
        if ocode != code or odev != dev or list(olens) != list(numels):
            raise ValueError("out must hold tensors of the lengths and type of grads")
    _raise(lib.b2g_clip_grad_norm(code, n, ptrs, numels, max_norm, optrs, norm.data_ptr(), p, nb,
                                  on.handle))
    on.uses(*grads, *outs)
    return norm
