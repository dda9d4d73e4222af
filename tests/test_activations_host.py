"""RMS norm and 8-bit activations: argument checks without a device, and the refusals of
the tensor calls.  The pointers below are never dereferenced."""
import ctypes

import pytest
import torch

P = 0x100000  # an aligned address
LONG = (1 << 31) - (1 << 16) + 1


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


@pytest.mark.parametrize("change,code", [
    ({"dtype": 2}, -12), ({"rows": -1}, -1), ({"cols": -1}, -1), ({"rows": 1 << 31}, -1),
    ({"cols": LONG, "ldx": LONG}, -1), ({"eps": -1.0}, -1), ({"eps": float("nan")}, -1),
    ({"ldx": 7}, -2), ({"ldr": 7}, -2), ({"ldt": 7}, -2), ({"ldy": 7}, -2), ({"ldyq": 7}, -2),
    ({"ldys": 0}, -2), ({"ldtq": 7}, -2), ({"ldts": 0}, -2), ({"x": None}, -3), ({"yq": None}, -3),
    ({"ts": None}, -3), ({"rows": 0, "x": None}, 0), ({"cols": 0, "x": None}, 0),
])
def test_rmsnorm_arguments(lib, change, code):
    a = dict(dtype=0, rows=4, cols=8, x=P, ldx=8, res=P, ldr=8, w=P, eps=1e-5, total=P, ldt=8, y=P,
             ldy=8, yq=P, ldyq=8, ys=P, ldys=1, tq=P, ldtq=8, ts=P, ldts=1, rstd=P, stream=0)
    a.update(change)
    assert lib.b2g_rmsnorm(*a.values()) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 2}, -12), ({"rows": -1}, -1), ({"cols": LONG}, -1), ({"lddy": 7}, -2), ({"ldt": 7}, -2),
    ({"lds": 0}, -2), ({"lddt": 7}, -2), ({"lddx": 7}, -2), ({"dy": None}, -3), ({"total": None}, -3),
    ({"rstd": None}, -3), ({"dx": None}, -3), ({"cols": 0}, 0), ({"rows": 0, "dw": None}, 0),
])
def test_rmsnorm_backward_arguments(lib, change, code):
    a = dict(dtype=0, rows=4, cols=8, dy=P, lddy=8, total=P, ldt=8, scales=P, lds=1, w=P, rstd=P,
             dtotal=P, lddt=8, dx=P, lddx=8, dw=P, ws=P, bytes=1 << 20, stream=0)
    a.update(change)
    assert lib.b2g_rmsnorm_backward(*a.values()) == code


@pytest.mark.parametrize("call", ["b2g_quantize8", "b2g_dequantize8"])
@pytest.mark.parametrize("change,code", [
    ({"dtype": 2}, -12), ({"rows": -1}, -1), ({"cols": LONG}, -1), ({"ldx": 7}, -2), ({"ldq": 7}, -2),
    ({"lds": 0}, -2), ({"x": None}, -3), ({"q": None}, -3), ({"s": None}, -3), ({"rows": 0}, 0),
    ({"cols": 0, "q": None}, 0),
])
def test_eightbit_arguments(lib, call, change, code):
    a = dict(dtype=0, rows=4, cols=8, x=P, ldx=8, q=P, ldq=8, s=P, lds=1)
    a.update(change)
    v = list(a.values())
    if call == "b2g_dequantize8":  # codes and scales first
        v = v[:3] + v[5:] + v[3:5]
    assert getattr(lib, call)(*v, 0) == code


@pytest.mark.parametrize("change,code", [
    ({"dtype": 2}, -12), ({"tokens": -1}, -1), ({"outs": -1}, -1), ({"width": -1}, -1),
    ({"tokens": LONG}, -1), ({"outs": LONG}, -1), ({"width": LONG}, -1), ({"lddy": 9}, -2),
    ({"ldq": 7}, -2), ({"lds": 0}, -2), ({"lddw": 7}, -2), ({"dy": None}, -3), ({"q": None}, -3),
    ({"s": None}, -3), ({"dw": None}, -3), ({"outs": 0}, 0), ({"width": 0}, 0),
    ({"tokens": 0, "acc": 1}, 0),
])
def test_weight_gradient_arguments(lib, change, code):
    a = dict(dtype=1, tokens=4, outs=10, width=8, dy=P, lddy=10, q=P, ldq=8, s=P, lds=1, acc=0, dw=P,
             lddw=8, ws=P, bytes=1 << 30, stream=0)
    a.update(change)
    assert lib.b2g_linear_dweight8(*a.values()) == code


def test_workspace_queries(lib):
    n = ctypes.c_size_t(99)
    q = lib.b2g_rmsnorm_backward_workspace_size
    assert q(5, 4, 8, ctypes.byref(n)) == -12 and q(0, 4, 8, None) == -3
    assert q(0, 4, 8, ctypes.byref(n)) == 0 and n.value >= 8 * 4
    q = lib.b2g_linear_dweight8_workspace_size
    assert q(5, 4, 8, 8, P, 8, ctypes.byref(n)) == -12 and q(0, 4, 8, 8, P, 8, None) == -3
    assert q(0, 4, 8, -8, P, 8, ctypes.byref(n)) == -1
    for dims in ((0, 8, 8), (4, 0, 8), (4, 8, 0)):
        assert q(1, *dims, P, 8, ctypes.byref(n)) == 0 and n.value == 0


def test_no_gpu_means_loud_failure(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.b2g_rmsnorm(0, 4, 8, P, 8, None, 0, P, 1e-5, None, 0, P, 8, None, 0, None, 0, None, 0,
                           None, 0, P, 0) == -5
    assert lib.b2g_quantize8(0, 4, 8, P, 8, P, 8, P, 1, 0) == -5
    assert lib.b2g_linear_dweight8(1, 4, 8, 8, P, 8, P, 8, P, 1, 0, P, 8, P, 1 << 30, 0) == -5


def test_tensor_calls_refuse(b2g):
    f = torch.zeros(4, 8)
    q, s = torch.zeros(4, 8, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.float8_e8m0fnu)
    for call in (lambda: b2g.rms_norm(f), lambda: b2g.rms_norm_8bit(f.half()),
                 lambda: b2g.quantize_8bit(f), lambda: b2g.quantize_8bit(3),
                 lambda: b2g.dequantize_8bit(q, s), lambda: b2g.dequantize_8bit(f, s),
                 lambda: b2g.rms_norm_backward(f, f, None, f[:, 0]),
                 lambda: b2g.linear_weight_grad_8bit(f, q, s)):
        with pytest.raises(TypeError):
            call()


def test_lengths_are_not_cut(b2g):
    """A length of 2^32 + 5 must not reach the library as 5."""
    with pytest.raises(b2g.B2GError):
        b2g.activations._length(5, (1 << 32) + 5)


def test_form_of_the_helpers():
    """The definition in 64 bits that the GPU tests compare with, against torch's own
    conversion where that has to agree."""
    import eightbit_helpers as e8

    x = torch.randn(9, 70) * torch.exp(4 * torch.randn(9, 70))
    codes, scales = e8.encode(x)
    each = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :70]
    want = (x.double() / each).float().to(torch.float8_e4m3fn)
    assert torch.equal(codes, want.view(torch.uint8))
    v = e8.values(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu))
    assert torch.equal(v, want.double() * each)
    assert ((v - x).abs() <= torch.maximum(2.0 ** -4 * x.abs().double(), 2.0 ** -10 * each)).all()
    assert (v.abs() / each).max() <= 448


@pytest.mark.gpu
def test_tensor_calls_refuse_on_gpu(b2g):
    x = torch.zeros(6, 40, device="cuda")
    q, s = b2g.quantize_8bit(x)
    r, w = x[:, 0].contiguous(), x[0]
    bad = [
        lambda: b2g.quantize_8bit(x.t()), lambda: b2g.quantize_8bit(x[0].expand(6, 40)),
        lambda: b2g.dequantize_8bit(q, s[:, :1]), lambda: b2g.dequantize_8bit(q[:5], s),
        lambda: b2g.dequantize_8bit(q.t(), s), lambda: b2g.dequantize_8bit(q[0], s[0]),
        lambda: b2g.dequantize_8bit(q, s, torch.float32, out=x[:5]),
        lambda: b2g.rms_norm(x, w[:7]), lambda: b2g.rms_norm(x, w, x[:5]),
        lambda: b2g.rms_norm(x, out=x), lambda: b2g.rms_norm(x, out=x[:3]),
        lambda: b2g.rms_norm(x[:4], None, x[:4], out=x[1:5]),
        lambda: b2g.rms_norm_8bit(x.t()),
        lambda: b2g.rms_norm_backward(x, x[:5], w, r), lambda: b2g.rms_norm_backward(x, x, w, r[:5]),
        lambda: b2g.rms_norm_backward(x, (q[:5], s[:5]), w, r),
        lambda: b2g.rms_norm_backward(x, (q, s[:5]), w, r),
        lambda: b2g.rms_norm_backward(x, x, w[:3], r), lambda: b2g.rms_norm_backward(x, x, w, r, x[:5]),
        lambda: b2g.rms_norm_backward(x.clone(), x, w.clone(), r, out=x),
        lambda: b2g.linear_weight_grad_8bit(x[:5], q, s),
        lambda: b2g.linear_weight_grad_8bit(x, q, s, accumulate=True),
        lambda: b2g.linear_weight_grad_8bit(x, q, s, dw=x),
        lambda: b2g.linear_weight_grad_8bit(x.t()[:6], q, s),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: b2g.rms_norm(x, w.bfloat16()), lambda: b2g.rms_norm(x.double()),
                 lambda: b2g.rms_norm(x, w, x.bfloat16()), lambda: b2g.dequantize_8bit(x, s),
                 lambda: b2g.dequantize_8bit(q, x), lambda: b2g.dequantize_8bit(q, s, torch.float16),
                 lambda: b2g.rms_norm_backward(x, q, w, r), lambda: b2g.rms_norm_backward(x, 3, w, r),
                 lambda: b2g.rms_norm_backward(x, x.bfloat16(), w, r),
                 lambda: b2g.linear_weight_grad_8bit(x, x, s),
                 lambda: b2g.linear_weight_grad_8bit(x, q, s, dw=x.bfloat16())):
        with pytest.raises(TypeError):
            call()
    sixteen = torch.zeros(64, 40, device="cuda")
    kept = b2g.quantize_8bit(sixteen)
    square = sixteen[:40]
    with pytest.raises(ValueError, match="overlap"):
        b2g.linear_weight_grad_8bit(sixteen, *kept, dw=square)
    lib = b2g.train_library()
    args = (0, 6, 40, x.data_ptr(), 40, x.data_ptr(), 40, None, 0, w.data_ptr(), r.data_ptr(), None, 0,
            x.clone().data_ptr(), 40, w.clone().data_ptr())
    assert lib.b2g_rmsnorm_backward(*args, None, 0, 0) == b2g.B2G_ERR_WORKSPACE
