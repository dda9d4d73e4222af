"""Layer norm and its gradients on the GPU against the formulas in 64 bits."""
import pytest
import torch

from gpu_helpers import env
from train_helpers import TINY, U, close, directional, padded, untouched

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = U[F32]


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def gamma(cols):
    """Relative error of a row sum: a thread adds at most 64 values (or, in wide
    rows, cols / 512) one after another, then at most 16 levels of pairs."""
    return (64 + 16 + cols / 512) * U32


def gamma_rows(rows):
    """The same for a column sum: rows per block, blocks per adding warp, warps."""
    return (8 + rows / 152 + 1216 / 8 + 8) * U32


def forward64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd, xh


def forward_bounds(x, w, b, eps):
    """|mean| is off by gamma * mean|x|; the variance, a sum of squares of
    differences with that error in each, by (gamma + 4 U) of itself plus 2 |d| dm,
    which its square root halves; y then carries both errors times w."""
    y, mean, rstd, xh = forward64(x, w, b, eps)
    g = gamma(x.shape[1])
    dm = (g + U32) * x.double().abs().mean(1) + TINY
    dr = rstd * (g + 4 * U32 + dm * rstd) + TINY
    wa = 1 if w is None else w.double().abs()
    by = (dm * rstd)[:, None] * wa + (xh * wa).abs() * (dr / rstd)[:, None] \
        + 4 * U32 * (xh * wa).abs() + 2 * U32 * y.abs() + U[x.dtype] * y.abs() * (1 + 1e-6) + TINY
    return y, mean, rstd, by, dm, dr


SHAPES = [
    # rows, cols: one element, one warp's row, sizes around the chunk and block limits
    (1, 1), (3, 2), (5, 7), (1, 4096), (2, 31), (33, 32), (7, 129), (64, 256), (19, 1000),
    (40, 1025), (9, 2048), (700, 512), (305, 2049), (3, 4096), (610, 4096), (2, 8192), (31, 8193),
    (3, 16384), (2, 20001), (1217, 64), (5000, 96),
    # many rows: rings, aligned or not, up to their widest
    (700, 7), (2000, 33), (1300, 777), (900, 1025), (650, 4095), (640, 8192), (640, 8191),
    (620, 9001),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(b2g, rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows * 31 + cols)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, _ = padded(mk(rows, cols) * 1.5 + 0.7, dtype)
    dy, _ = padded(mk(rows, cols), dtype)
    w, b = (mk(cols) * 0.3 + 1).to(dtype).cuda(), mk(cols).to(dtype).cuda()
    y, mean, rstd = b2g.layer_norm(x, w, b, eps=1e-5)
    wy, wm, wr, by, dm, dr = forward_bounds(x, w, b, 1e-5)
    close(mean, wm, dm, "mean")
    close(rstd, wr, dr, "rstd")
    close(y, wy, by, "y")
    check_backward(b2g, dy, x, w, mean, rstd)


def check_backward(b2g, dy, x, w, mean, rstd, **kw):
    dtype, (rows, cols) = x.dtype, x.shape
    # the forward call's statistics are inputs here, so their own error is left out
    dx, dw, db = b2g.layer_norm_backward(dy, x, w, mean, rstd, **kw)
    X, D, m, r = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (X - m) * r
    g = D * (1 if w is None else w.double())
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    want = r * (g - c1 - xh * c2)
    k = gamma(cols) + 8 * U32
    bound = k * r * (g.abs() + g.abs().mean(1, keepdim=True)
                     + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
        + U[dtype] * want.abs() * (1 + 1e-6) + TINY
    close(dx, want, bound, "dx")
    k = gamma_rows(rows) + 4 * U32
    for got, part, what in ((dw, D * xh, "dweight"), (db, D, "dbias")):
        if got is not None:
            s = part.sum(0)
            close(got, s, k * part.abs().sum(0) + U[dtype] * s.abs() * (1 + 1e-6) + TINY, what)
    return dx, dw, db


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld_extra,offset", [(0, 1), (1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("cols", [64, 777, 4096])
def test_strides_alignment_and_guards(b2g, cols, ld_extra, offset, dtype):
    rows = 21
    gen = torch.Generator().manual_seed(cols + ld_extra)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, _ = padded(mk(rows, cols), dtype, cols + ld_extra, offset)
    w, b = mk(cols).to(dtype).cuda(), mk(cols).to(dtype).cuda()
    out, flat = padded(torch.zeros(rows, cols, dtype=torch.float64), dtype, cols + ld_extra + 2,
                       offset)
    before = flat.clone()
    y, mean, rstd = b2g.layer_norm(x, w, b, out=out)
    assert y is out and untouched(flat, out, before)
    close(y, *[forward_bounds(x, w, b, 1e-5)[i] for i in (0, 3)], "y")
    dy, _ = padded(mk(rows, cols), dtype, cols + ld_extra, offset)
    before = flat.clone()
    check_backward(b2g, dy, x, w, mean, rstd, out=out)
    assert untouched(flat, out, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [512, 1001, 20000])
def test_in_place(b2g, cols, dtype):
    gen = torch.Generator().manual_seed(cols)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b = (t.to(dtype).cuda() for t in (mk(37, cols), mk(cols), mk(cols)))
    dy = mk(37, cols).to(dtype).cuda()
    y, mean, rstd = b2g.layer_norm(x, w, b)
    dx, dw, db = b2g.layer_norm_backward(dy, x, w, mean, rstd)
    x2, dy2 = x.clone(), dy.clone()
    assert torch.equal(b2g.layer_norm(x2, w, b, out=x2)[0], y)
    got = b2g.layer_norm_backward(dy2, x, w, mean, rstd, out=dy2)
    assert got[0] is dy2 and all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_weight_and_bias(b2g, dtype):
    x = (torch.randn(50, 640, dtype=torch.float64) + 3).to(dtype).cuda()
    y, mean, rstd = b2g.layer_norm(x)
    close(y, *[forward_bounds(x, None, None, 1e-5)[i] for i in (0, 3)], "y")
    dy = torch.randn(50, 640, dtype=torch.float64).to(dtype).cuda()
    dx, dw, db = check_backward(b2g, dy, x, None, mean, rstd, bias=False)
    assert dw is None and db is None


def test_large_mean_keeps_digits(b2g):
    """The variance is that of the differences: a mean 4000 times the spread
    costs no more than the rounding of x - mean."""
    x = (torch.randn(8, 1024, dtype=torch.float64) + 4096).float().cuda()
    y, mean, rstd = b2g.layer_norm(x)
    close(y, *[forward_bounds(x, None, None, 1e-5)[i] for i in (0, 3)], "y")


def test_constant_rows_and_nonfinite(b2g):
    x = torch.full((4, 300), 2.5, device="cuda")
    x[1, 7] = float("inf")
    x[2, 299] = float("nan")
    y, mean, rstd = b2g.layer_norm(x)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.equal(y[3], y[0])
    assert abs(float(rstd[0]) - 1e-5 ** -0.5) < 1e-3
    assert torch.isnan(y[1]).any() and torch.isnan(y[2]).all()


def test_no_rows(b2g):
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = b2g.layer_norm(x, w, w)
    dx, dw, db = b2g.layer_norm_backward(x, x, w, mean, rstd)
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()


def test_same_bits_every_run(b2g):
    x = torch.randn(3000, 1025, device="cuda")
    w, b = torch.randn(1025, device="cuda"), torch.randn(1025, device="cuda")
    y, mean, rstd = b2g.layer_norm(x, w, b)
    first = b2g.layer_norm_backward(y, x, w, mean, rstd)
    for _ in range(5):
        assert all(torch.equal(p, q)
                   for p, q in zip(first, b2g.layer_norm_backward(y, x, w, mean, rstd)))


def test_gradient_against_differences(b2g):
    """d/dt sum(dy * y(x + t u)) and the same in the weight and bias, by central
    differences of the forward call itself."""
    torch.manual_seed(3)
    x, w, b, dy = (torch.randn(*s, device="cuda") for s in ((12, 96), (96,), (96,), (12, 96)))
    _, mean, rstd = b2g.layer_norm(x, w, b)
    grads = b2g.layer_norm_backward(dy, x, w, mean, rstd)
    eps = 2.0 ** -7
    for k, g in enumerate(grads):
        u = torch.randn_like((x, w, b)[k])

        def loss(t):
            args = [x, w, b]
            args[k] = args[k] + t * u
            return float((b2g.layer_norm(*args)[0].double() * dy.double()).sum())

        diff, trunc = directional(loss, eps)
        by = forward_bounds(x, w, b, 1e-5)[3]
        # both ends carry the forward's error and that of forming x + t u
        noise = float((dy.double().abs() * (by + 8 * U32)).sum()) * 4 / eps
        want = float((g.double() * u.double()).sum())
        assert abs(diff - want) <= trunc + noise, (k, diff, want, trunc, noise)


def test_other_stream(b2g):
    x = torch.randn(512, 2048, device="cuda")
    ref = b2g.layer_norm(x)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, mean, rstd = b2g.layer_norm(x, stream=s)
    dx, _, _ = b2g.layer_norm_backward(x, x, None, mean, rstd, stream=s)
    s.synchronize()
    assert torch.equal(y, ref) and bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("cols", [2048, 2040, 2047])
def test_bounded_waits_of_the_rings(b2g, cols):
    """With each group's copies stopped after one row the waits run out, the calls return
    and the status word says so; the next calls work again."""
    x = torch.randn(8192, cols, device="cuda").bfloat16()
    w = torch.randn(cols, device="cuda").bfloat16()
    stream = torch.cuda.current_stream().cuda_stream

    def forward():
        return b2g.layer_norm(x, w, w)

    y, mean, rstd = forward()

    def backward():
        return b2g.layer_norm_backward(y, x, w, mean, rstd)

    for call in (forward, backward) if cols % 8 == 0 else (backward,):  # odd rows: one ring
        first = call()
        torch.cuda.synchronize()
        try:
            b2g.b2g_set_wait_limit_ns(2_000_000)
            b2g.b2g_debug_stop_after(1)
            call()
            rc, flags = b2g.b2g_status(stream)
            assert rc == b2g.B2G_ERR_TIMEOUT and flags & 1 and flags & 4
        finally:
            b2g.b2g_debug_stop_after(-1)
            b2g.b2g_set_wait_limit_ns(2_000_000_000)
        again = call()
        assert all(torch.equal(p, q) for p, q in zip(first, again))
        assert b2g.b2g_status(stream) == (0, 0)


@pytest.mark.parametrize("side", [False, True])
def test_no_columns(b2g, side):
    """Rows of nothing have no mean: NaN, not what the memory held."""
    stream = torch.cuda.Stream() if side else None
    x = torch.empty(1000, 0, device="cuda")
    junk = [torch.full((1000,), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del junk  # the allocator hands these out again
    y, mean, rstd = b2g.layer_norm(x, stream=stream)
    dx, dw, db = b2g.layer_norm_backward(x, x, x[0], mean, rstd, stream=stream)
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (1000, 0) and dw.shape == db.shape == (0,)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
