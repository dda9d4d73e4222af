"""include/b2g_train.h: every declared call is exported, and the argument checks
answer with the documented codes before anything reaches a device.  The
pointers below are never dereferenced."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "b2g_train.h")
P = 0x100000  # an aligned address


@pytest.fixture(scope="module")
def b2g():
    from dense_fp32_gemm_07_gb300 import build

    build.build()
    import dense_fp32_gemm_07_gb300 as pkg

    pkg.train_library()
    return pkg


@pytest.fixture(scope="module")
def lib(b2g):
    return b2g.train_library()


def test_declared_calls_are_exported(b2g):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(b2g_\w+)\s*\(", text)))
    assert names == sorted(b2g.TRAIN_EXPORTS)
    raw = ctypes.CDLL(b2g.LIB_PATH)
    assert all(hasattr(raw, n) for n in names)


def test_codes_match_header(b2g):
    for name, val in re.findall(r"#define (B2G_\w+) \(?(-?\d+)\)?", open(HEADER).read()):
        assert getattr(b2g, name) == int(val), name
        if int(val) < 0:
            assert b2g.b2g_strerror(int(val)) != "unknown error code"


def size(query, *args):
    n = ctypes.c_size_t(99)
    return query(*args, ctypes.byref(n)), n.value


@pytest.mark.parametrize("change,code", [
    ({"dtype": 2}, -12), ({"rows": -1}, -1), ({"cols": -1}, -1), ({"eps": -1.0}, -1),
    ({"eps": float("nan")}, -1), ({"ldx": 7}, -2), ({"ldy": 7}, -2), ({"x": None}, -3),
    ({"y": None}, -3), ({"rows": 0, "x": None}, 0), ({"cols": 0, "x": None}, 0),
    ({"rows": 1 << 31}, -1),
])
def test_layernorm_arguments(lib, change, code):
    a = dict(dtype=0, rows=4, cols=8, x=P, ldx=8, w=P, b=P, eps=1e-5, y=P, ldy=8, mean=P, rstd=P,
             stream=0)
    a.update(change)
    assert lib.b2g_layernorm(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": -1}, -12), ({"rows": -1}, -1), ({"lddy": 7}, -2), ({"ldx": 7}, -2),
    ({"lddx": 7}, -2), ({"dy": None}, -3), ({"mean": None}, -3), ({"dx": None}, -3),
    ({"cols": 0}, 0), ({"rows": 0, "dw": None, "db": None}, 0),
])
def test_layernorm_backward_arguments(lib, change, code):
    a = dict(dtype=0, rows=4, cols=8, dy=P, lddy=8, x=P, ldx=8, w=P, mean=P, rstd=P, dx=P, lddx=8,
             dw=P, db=P, ws=P, bytes=1 << 20, stream=0)
    a.update(change)
    assert lib.b2g_layernorm_backward(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 3}, -12), ({"id_bytes": 2}, -12), ({"tokens": -1}, -1), ({"vocab": -1}, -1),
    ({"width": -1}, -1), ({"ldt": 7}, -2), ({"ldo": 7}, -2), ({"ids": None}, -3),
    ({"out": None}, -3), ({"tokens": 0, "ids": None}, 0), ({"width": 0}, 0),
    ({"tokens": (1 << 30) + 1}, -1),
])
def test_embedding_arguments(lib, change, code):
    a = dict(dtype=0, tokens=4, vocab=10, width=8, ids=P, id_bytes=8, table=P, ldt=8, scale=1.0,
             out=P, ldo=8, stream=0)
    a.update(change)
    assert lib.b2g_embedding(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 3}, -12), ({"id_bytes": 1}, -12), ({"tokens": -1}, -1), ({"ldd": 7}, -2),
    ({"ldt": 7}, -2), ({"dtable": None}, -3), ({"ids": None}, -3), ({"vocab": 0}, 0),
    ({"width": 0}, 0), ({"tokens": 0, "acc": 1}, 0),
])
def test_embedding_backward_arguments(lib, change, code):
    a = dict(dtype=0, tokens=4, vocab=10, width=8, ids=P, id_bytes=8, dout=P, ldd=8, scale=1.0,
             pad=-1, acc=0, dtable=P, ldt=8, ws=P, bytes=1 << 30, stream=0)
    a.update(change)
    assert lib.b2g_embedding_backward(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 3}, -12), ({"id_bytes": 1}, -12), ({"tokens": -1}, -1), ({"vocab": 0}, -1),
    ({"width": 0}, -1), ({"ldh": 7}, -2), ({"ldw": 7}, -2), ({"h": None}, -3), ({"w": None}, -3),
    ({"target": None}, -3), ({"lse": None}, -3), ({"tokens": 0, "h": None}, 0),
])
def test_linear_xent_arguments(lib, change, code):
    a = dict(dtype=1, tokens=4, vocab=10, width=8, h=P, ldh=8, w=P, ldw=8, target=P, id_bytes=8,
             ignore=-100, loss=P, lse=P, ws=P, bytes=1 << 30, stream=0)
    a.update(change)
    assert lib.b2g_linear_xent(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 3}, -12), ({"id_bytes": 1}, -12), ({"tokens": -1}, -1), ({"vocab": 0}, -1),
    ({"ldh": 7}, -2), ({"ldw": 7}, -2), ({"lddh": 7}, -2), ({"lddw": 7}, -2), ({"h": None}, -3),
    ({"lse": None}, -3), ({"gloss": None}, -3), ({"dh": None, "dw": None}, 0),
    ({"tokens": 0, "acc": 1}, 0), ({"tokens": 0, "dw": None}, 0),
])
def test_linear_xent_backward_arguments(lib, change, code):
    a = dict(dtype=1, tokens=4, vocab=10, width=8, h=P, ldh=8, w=P, ldw=8, target=P, id_bytes=8,
             ignore=-100, lse=P, gloss=P, dh=P, lddh=8, acc=0, dw=P, lddw=8, ws=P, bytes=1 << 30,
             stream=0)
    a.update(change)
    assert lib.b2g_linear_xent_backward(*a.values()) == code


LONG = (1 << 31) - (1 << 16) + 1


def test_lengths_past_the_limits(lib):
    """Refused before anything else of the call is looked at."""
    n = ctypes.c_size_t()
    assert lib.b2g_layernorm(0, 4, LONG, P, LONG, P, P, 1e-5, P, LONG, P, P, 0) == -1
    assert lib.b2g_layernorm_backward_workspace_size(0, 4, LONG, ctypes.byref(n)) == -1
    for vocab, width in ((LONG, 8), (8, LONG)):
        assert lib.b2g_embedding(0, 4, vocab, width, P, 8, P, LONG, 1.0, P, LONG, 0) == -1
        assert lib.b2g_embedding_backward_workspace_size(0, 4, vocab, width, ctypes.byref(n)) == -1
    for tokens, vocab, width in ((LONG, 8, 8), (8, LONG, 8), (8, 8, LONG)):
        assert lib.b2g_linear_xent_workspace_size(1, tokens, vocab, width, P, LONG, P, LONG, 0,
                                                  ctypes.byref(n)) == -1


def test_clip_arguments(lib):
    one, n = (ctypes.c_void_p * 1)(P), (ctypes.c_longlong * 1)(5)
    neg, null = (ctypes.c_longlong * 1)(-5), (ctypes.c_void_p * 1)(None)
    clip, norm = lib.b2g_clip_grad_norm, lib.b2g_grad_norm
    assert norm(7, 1, one, n, P, P, 1 << 20, 0) == -12
    assert norm(0, -1, one, n, P, P, 1 << 20, 0) == -1
    assert norm(0, 1, one, neg, P, P, 1 << 20, 0) == -1
    assert norm(0, 1, null, n, P, P, 1 << 20, 0) == -3
    assert norm(0, 1, None, n, P, P, 1 << 20, 0) == -3
    assert norm(0, 1, one, n, None, P, 1 << 20, 0) == -3
    assert clip(0, 1, one, n, -1.0, one, P, P, 1 << 20, 0) == -1
    assert clip(0, 1, one, n, float("nan"), one, P, P, 1 << 20, 0) == -1
    assert clip(0, 1, one, n, 1.0, None, P, P, 1 << 20, 0) == -3
    assert clip(0, 1, one, n, 1.0, null, P, P, 1 << 20, 0) == -3


def test_workspace_queries(lib):
    assert size(lib.b2g_layernorm_backward_workspace_size, 5, 4, 8)[0] == -12
    assert lib.b2g_layernorm_backward_workspace_size(0, 4, 8, None) == -3
    rc, n = size(lib.b2g_layernorm_backward_workspace_size, 0, 4, 8)
    assert rc == 0 and n >= 2 * 8 * 4 and n % 64 == 0  # whole pairs of partial rows
    assert size(lib.b2g_embedding_backward_workspace_size, 0, 0, 10, 8) == (0, 0)
    rc, n = size(lib.b2g_embedding_backward_workspace_size, 1, 1000, 10, 8)
    assert rc == 0 and n > 4 * 4 * 1000  # two copies of ids and places, counts, partial rows
    q = lib.b2g_linear_xent_workspace_size
    assert size(q, 1, 4, 10, 0, P, 8, P, 8, 0)[0] == -1 and q(1, 4, 10, 8, P, 8, P, 8, 0, None) == -3
    assert size(q, 1, 0, 10, 8, P, 8, P, 8, 1) == (0, 0)
    fwd = size(q, 1, 128, 1000, 128, P, 128, P, 128, 0)[1]
    assert 0 < fwd < 128 * 1000 * 4         # less than the logits
    # an operand off the 16-byte boundaries is copied, FP32 ones become three planes
    assert size(q, 1, 128, 1000, 128, P, 128, P + 2, 128, 0)[1] == fwd + 1000 * 128 * 2
    assert size(q, 0, 128, 1000, 128, P, 128, P, 128, 0)[1] == fwd + 3 * 1128 * 128 * 2
    # up to 64 tokens FP32's w is read as it is: only h becomes planes
    few = size(q, 1, 64, 1000, 128, P, 128, P, 128, 0)[1]
    assert size(q, 0, 64, 1000, 128, P, 128, P, 128, 0)[1] == few + 3 * 64 * 128 * 2
    # dz exists a piece at a time: a larger vocabulary needs no more room for it
    big = [size(q, 1, 8192, v, 512, P, 512, P, 512, 1)[1] for v in (65536, 1 << 20)]
    assert big[1] <= big[0] < (1 << 30)
    lens = (ctypes.c_longlong * 3)(1, 0, 1 << 40)
    rc, n = size(lib.b2g_grad_norm_workspace_size, 0, 3, lens)
    assert rc == 0 and 4 <= n <= 4 * 152 * 4 * 4
    assert size(lib.b2g_grad_norm_workspace_size, 0, 0, None) == (0, 4)


def test_no_gpu_means_loud_failure(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    n = (ctypes.c_longlong * 1)(5)
    one = (ctypes.c_void_p * 1)(P)
    assert lib.b2g_layernorm(0, 4, 8, P, 8, P, P, 1e-5, P, 8, P, P, 0) == -5
    assert lib.b2g_embedding(0, 4, 10, 8, P, 8, P, 8, 1.0, P, 8, 0) == -5
    assert lib.b2g_grad_norm(0, 1, one, n, P, P, 1 << 20, 0) == -5
    assert lib.b2g_linear_xent(1, 4, 10, 8, P, 8, P, 8, P, 8, -100, P, P, P, 1 << 30, 0) == -5


def test_tensor_calls_refuse(b2g):
    f = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        b2g.layer_norm(f)  # not on a GPU
    with pytest.raises(TypeError):
        b2g.layer_norm(f.half())
    with pytest.raises(TypeError):
        b2g.embedding(torch.zeros(3), f)
    with pytest.raises(ValueError):
        b2g.clip_grad_norm([f], -1.0)
    with pytest.raises(ValueError):
        b2g.grad_norm([])


BUILD_ALONE = """
import os, sys
sys.path.insert(0, sys.argv[1])
from dense_fp32_gemm_07_gb300 import build as b
out, how = sys.argv[2:]
b.BUILD, b.LIB = os.path.join(out, "build"), os.path.join(out, "libb2g_sgemm.so")
b.BINDING = os.path.join(out, "_train_binding.so")
b.sources = lambda: ["noalloc.cu"]     # one small file stands for all
if how == "hidden":
    sys.modules["torch"] = None        # as where it is not installed
else:
    b.shutil.which = lambda name, which=b.shutil.which: "/bin/false" if name == "g++" else which(name)
assert not b.up_to_date()
try:
    assert b.build() == b.LIB and how == "hidden"
    assert b.up_to_date() and "torch" not in [m for m in sys.modules if sys.modules[m]]
except RuntimeError as e:
    assert how == "broken" and "train_binding.cpp" in str(e), e
    assert not b.up_to_date()
assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
"""


@pytest.mark.parametrize("how", ["hidden", "broken"])
def test_library_builds_without_the_binding(tmp_path, how):
    """Without torch the C library is built alone; a binding that fails is reported, with
    the library linked all the same."""
    subprocess.run([sys.executable, "-c", BUILD_ALONE, ROOT, str(tmp_path), how], check=True)


def test_another_torch_makes_the_binding_stale(b2g, monkeypatch, tmp_path):
    from dense_fp32_gemm_07_gb300 import build

    assert build.up_to_date()
    monkeypatch.setattr(build, "_torch_stamp", lambda: "0.0 elsewhere")
    assert not build.up_to_date()
    monkeypatch.setattr(build, "_torch_stamp", lambda: None)
    assert build.up_to_date()


def test_results_beside_their_inputs(b2g):
    """Columns of one buffer that share no element may be result and input; a shared
    column, row or element may not."""
    apart = b2g.train._apart
    flat = torch.zeros(6 * 24 + 40)
    buf = flat[:144].view(6, 24)
    left, right, middle = buf[:, :8], buf[:, 8:20], buf[:, 7:9]
    for out, x in ((left, right), (right, left), (buf[:, 20:], left), (left[2:], right[:5]),
                   (left, right[1:]), (buf[:3], buf[3:]), (left, flat[140:170])):
        apart(out, ("x", x))
    shifted = flat[20:20 + 120].view(5, 24)[:, :8]   # columns 20 .. 23, then 0 .. 3 of the next row
    for out, x in ((left, left), (left, middle), (right, middle), (left, shifted), (shifted, left),
                   (buf, left), (left, flat[3:30]), (left, flat[:144].view(18, 8)[3:5]),
                   (left[:1], left[:1])):
        with pytest.raises(ValueError):
            apart(out, ("x", x))
    apart(buf[:, 12:20], ("x", shifted))
    half = torch.zeros(4, 32, dtype=torch.bfloat16)
    apart(half[:, 16:], ("x", half[:, :16]))
    with pytest.raises(ValueError):
        apart(half[:, 15:], ("x", half[:, :16]))


@pytest.mark.gpu
def test_result_beside_its_input_on_gpu(b2g):
    """Each call with a given result, whose rows lie between its input's rows."""
    torch.manual_seed(0)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.randn(300, 160, device="cuda").to(dt)
        x, out = buf[:, :80], buf[:, 80:]
        w = torch.randn(80, device="cuda").to(dt)
        y, mean, rstd = b2g.layer_norm(x.contiguous(), w, w)
        assert torch.equal(b2g.layer_norm(x, w, w, out=out)[0], y) and torch.equal(out, y)
        dx = b2g.layer_norm_backward(y, x.contiguous(), w, mean, rstd)[0]
        got = b2g.layer_norm_backward(y, x, w, mean, rstd, out=out)[0]
        assert torch.equal(got, dx)
        ids = torch.arange(300, device="cuda").flip(0)
        want = b2g.embedding(ids, x.contiguous())
        assert torch.equal(b2g.embedding(ids, x, out=out), want)
        want = b2g.embedding_backward(ids, x.contiguous(), 300)
        assert torch.equal(b2g.embedding_backward(ids, x, 300, out=out), want)
        h, t = torch.randn(100, 80, device="cuda").to(dt), ids[:100].contiguous()
        _, lse = b2g.linear_cross_entropy(h, x, t)
        g = torch.full((100,), 0.01, device="cuda")
        keep = x.clone()
        want = b2g.linear_cross_entropy_backward(h, keep, t, lse, g)
        got = b2g.linear_cross_entropy_backward(h, x, t, lse, g, dw=out)
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(x, keep)


@pytest.mark.gpu
def test_tensor_calls_refuse_on_gpu(b2g):
    x = torch.zeros(6, 8, device="cuda")
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    bad = [
        lambda: b2g.layer_norm(x.t()), lambda: b2g.layer_norm(x, x[0, :7]),
        lambda: b2g.layer_norm(x, out=x[:3]), lambda: b2g.layer_norm(x[:4], out=x[1:5]),
        lambda: b2g.layer_norm(x[0].expand(6, 8)),
        lambda: b2g.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
        lambda: b2g.layer_norm_backward(x[:5], x, None, x[0, :6], x[0, :6]),
        lambda: b2g.embedding(ids[::2], x), lambda: b2g.embedding(ids, x, out=x),
        lambda: b2g.embedding_backward(ids[:5], x, 10),
        lambda: b2g.embedding_backward(ids, x, 10, accumulate=True),
        lambda: b2g.embedding_backward(ids, x, 10, padding_idx=10),
        lambda: b2g.embedding_backward(ids, x, 6, out=x),
        lambda: b2g.linear_cross_entropy(x, x[:, :7], ids),
        lambda: b2g.linear_cross_entropy(x, x, ids[:5]),
        lambda: b2g.linear_cross_entropy_backward(x, x, ids, x[0, :6], x[0, :5]),
        lambda: b2g.linear_cross_entropy_backward(x, x, ids, x[0, :6], x[0, :6], dw=x),
        lambda: b2g.linear_cross_entropy_backward(x, x, ids, x[0, :6], x[0, :6], accumulate=True),
        lambda: b2g.clip_grad_norm([x.t()], 1.0),
        lambda: b2g.clip_grad_norm([x], 1.0, out=[x[:5]]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: b2g.layer_norm(x, x[0].bfloat16()), lambda: b2g.layer_norm(x.double()),
                 lambda: b2g.embedding(ids.float(), x),
                 lambda: b2g.grad_norm([x, x.bfloat16()])):
        with pytest.raises(TypeError):
            call()
    n = ctypes.c_size_t(0)
    lib = b2g.train_library()
    args = (0, 6, 8, x.data_ptr(), 8, x.data_ptr(), 8, None, x.data_ptr(), x.data_ptr(),
            x.data_ptr(), 8, x.data_ptr(), None)
    assert lib.b2g_layernorm_backward(*args, None, 0, 0) == b2g.B2G_ERR_WORKSPACE
    lib.b2g_layernorm_backward_workspace_size(0, 6, 8, ctypes.byref(n))
    ws = torch.empty(n.value + 16, dtype=torch.uint8, device="cuda")
    assert lib.b2g_layernorm_backward(*args, ws.data_ptr(), n.value - 1, 0) == b2g.B2G_ERR_WORKSPACE
    assert lib.b2g_layernorm_backward(*args, ws.data_ptr() + 4, n.value, 0) == b2g.B2G_ERR_WORKSPACE


@pytest.mark.gpu
def test_results_over_smaller_inputs_are_refused(b2g):
    """A result must not overlap a call's vectors either: other rows still read them."""
    x = torch.ones(6, 8, device="cuda")
    buf = torch.ones(200, device="cuda")
    out, part = buf[:48].view(6, 8), buf[40:48]
    six, n = buf[44:50], x[:, 0].contiguous()
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    bad = [
        lambda: b2g.layer_norm(x, part, out=out), lambda: b2g.layer_norm(x, None, part, out=out),
        lambda: b2g.layer_norm_backward(x, x, part, n, n, out=out),
        lambda: b2g.layer_norm_backward(x, x, None, six, n, out=out),
        lambda: b2g.layer_norm_backward(x, x, None, n, six, out=out),
        lambda: b2g.linear_cross_entropy_backward(x, x, ids, six, n, dw=out),
        lambda: b2g.linear_cross_entropy_backward(x, x, ids, n, six, dw=out),
        lambda: b2g.linear_cross_entropy_backward(x, x, out.view(torch.int64).view(-1)[:6], n, n,
                                                  dw=out),
    ]
    for call in bad:
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert (buf == 1).all()
