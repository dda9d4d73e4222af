"""RMS norm with residual and 8-bit results, and its gradients, against 64 bits."""
import pytest
import torch

import eightbit_helpers as e8
from gpu_helpers import env
from train_helpers import TINY, U, close, directional, padded, untouched

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = U[F32]
EPS = 1e-5


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def gamma(cols):
    """Relative error of a row's sum of terms' absolute values: a thread adds at most 64 of
    them (or, in wide rows, cols / 512) one after another, then at most 16 levels of pairs."""
    return (64 + 16 + cols / 512) * U32


def gamma_rows(rows):
    """The same for a column sum: rows per block, blocks per adding warp, warps."""
    return (8 + rows / 152 + 1216 / 8 + 8) * U32


def check_forward(x, res, w, y, total, rstd):
    """total is one rounding; rstd the square root of a sum of squares that is within gamma
    of itself; y carries that and two products' roundings, then its own."""
    dtype = x.dtype
    if res is None:
        assert total is x
    else:
        assert torch.equal(total, (x.float() + res.float()).to(dtype))
    t = total.double()
    want = 1 / torch.sqrt(t.square().mean(1) + EPS)
    rel = gamma(x.shape[1]) / 2 + 4 * U32
    close(rstd, want, want * rel + TINY, "rstd")
    want_y = t * want[:, None] * (1 if w is None else w.double())
    dy = want_y.abs() * (rel + 4 * U32) + TINY  # in FP32
    if y is not None:
        close(y, want_y, dy + U[dtype] * want_y.abs() * (1 + 1e-4) + TINY, "y")
    return want_y, dy


def check_y8(y8, want, dy):
    """Scales of the exact largest values, or of those an FP32 error away from them; codes
    within half a step: 2^-4 of a value, or 2^-10 of the scale."""
    v = e8.values(*y8)
    s = torch.exp2(y8[1].cpu().contiguous().view(torch.uint8).double() - 127)
    want, dy = want.cpu(), dy.cpu()
    pad = (0, s.shape[1] * 32 - want.shape[1])
    blocks = lambda a: torch.nn.functional.pad(a, pad).view(len(a), -1, 32).amax(2)  # noqa: E731
    lo, hi = blocks(want.abs() - dy), blocks(want.abs() + dy)
    for side, ok in ((lo, torch.ge), (hi, torch.le)):
        e = torch.tensor([[e8.exponent(max(0.0, float(a))) for a in row] for row in side],
                         dtype=torch.float64)
        assert ok(s, torch.exp2(e)).all()
    each = s.repeat_interleave(32, 1)[:, :want.shape[1]]
    close(v, want, dy * 1.1 + torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * each), "y8")


def check_backward(b2g, dy, total, w, rstd, dtotal, **kw):
    dx, dw = b2g.rms_norm_backward(dy, total, w, rstd, dtotal=dtotal, **kw)
    dtype, (rows, cols) = dy.dtype, dy.shape
    T = e8.values(*total).cuda() if isinstance(total, tuple) else total.double()
    D, r = dy.double(), rstd.double()[:, None]
    xh = T * r
    g = D * (1 if w is None else w.double())
    c = (g * xh).mean(1, keepdim=True)
    own = r * (g - xh * c)
    want = own + (0 if dtotal is None else dtotal.double())
    k = gamma(cols) + 8 * U32
    bound = k * r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) \
        + 2 * U32 * want.abs() + U[dtype] * want.abs() * (1 + 1e-4) + TINY
    close(dx, want, bound, "dx")
    if w is None:
        assert dw is None
    else:
        part = D * xh
        s = part.sum(0)
        close(dw, s, (gamma_rows(rows) + 4 * U32) * part.abs().sum(0) + U[dtype] * s.abs() * (1 + 1e-4)
              + TINY, "dweight")
    return dx, dw


SHAPES = [
    (1, 1), (3, 2), (5, 7), (1, 4096), (2, 31), (33, 32), (7, 129), (64, 256), (19, 1000),
    (40, 1025), (9, 2048), (700, 512), (305, 2049), (610, 4096), (2, 8192), (31, 8193),
    (3, 16384), (2, 20001), (1217, 64), (5000, 96), (128, 4096), (1000, 5120),
    (700, 7), (2000, 33), (1300, 777), (900, 1025), (650, 4095), (640, 8192), (640, 8191),
    (620, 9001), (1500, 1032), (4000, 2048), (9000, 40), (3000, 512), (3000, 528), (2500, 3000),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(b2g, rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows * 31 + cols)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, res = (mk(rows, cols).to(dtype).cuda() for _ in range(2))
    dy, dtotal = (mk(rows, cols).to(dtype).cuda() for _ in range(2))
    w = (mk(cols) * 0.3 + 1).to(dtype).cuda()
    y, total, rstd = b2g.rms_norm(x, w, res, EPS)
    want, dy32 = check_forward(x, res, w, y, total, rstd)
    got = b2g.rms_norm_8bit(x, w, res, EPS, with_y=True, keep_total=True)
    if cols * x.element_size() % 16 == 0:  # other rows are added up in another order
        assert torch.equal(got[0], y) and torch.equal(got[2], rstd)
    check_forward(x, res, w, *got[:3])
    check_y8(got[3], want, dy32)
    if dtype is F32:  # y is what was rounded to 8 bits
        assert all(e8.same_bytes(a, b) for a, b in zip(got[3], b2g.quantize_8bit(got[0])))
    assert all(e8.same_bytes(a, b) for a, b in zip(got[4], b2g.quantize_8bit(total)))
    check_backward(b2g, dy, total, w, rstd, dtotal)
    check_backward(b2g, dy, got[4], w, rstd, dtotal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(3, 4096), (16, 4096), (17, 4096), (2, 8192), (9, 8191),
                                       (63, 777), (64, 777), (65, 777), (129, 40), (1024, 40),
                                       (1025, 33), (640, 96)])
def test_backward_of_few_blocks(b2g, rows, cols, dtype):
    """dweight of 2 to 9 blocks: a cluster that adds its blocks' sums, or a launch that does."""
    gen = torch.Generator().manual_seed(rows + cols)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, dy, dtotal = (mk(rows, cols).to(dtype).cuda() for _ in range(3))
    w = (mk(cols) * 0.3 + 1).to(dtype).cuda()
    _, total, rstd = b2g.rms_norm(x, w)
    kept = b2g.quantize_8bit(total)
    for held in (total, kept):
        check_backward(b2g, dy, held, w, rstd, dtotal)
        check_backward(b2g, dy, held, w, rstd, None)
        one, two = (b2g.rms_norm_backward(dy, held, w, rstd, dtotal) for _ in range(2))
        assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(50, 640), (30, 333), (2000, 1024), (1500, 333), (5, 9001)])
def test_without_weight_and_residual(b2g, rows, cols, dtype):
    x = (torch.randn(rows, cols, dtype=torch.float64) + 3).to(dtype).cuda()
    y, total, rstd = b2g.rms_norm(x)
    check_forward(x, None, None, y, total, rstd)
    none, total, rstd, y8, t8 = b2g.rms_norm_8bit(x)
    assert none is None and t8 is None and total is x
    check_y8(y8, *check_forward(x, None, None, None, total, rstd))
    kept = b2g.rms_norm_8bit(x, keep_total=True)[4]
    assert all(e8.same_bytes(a, b) for a, b in zip(kept, b2g.quantize_8bit(x)))
    if dtype is F32:
        got = b2g.rms_norm_8bit(x, with_y=True)
        assert all(e8.same_bytes(a, b) for a, b in zip(got[3], b2g.quantize_8bit(got[0])))
    dy = torch.randn(rows, cols, dtype=torch.float64).to(dtype).cuda()
    check_backward(b2g, dy, x, None, rstd, None)
    check_backward(b2g, dy, b2g.quantize_8bit(x), None, rstd, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld_extra,offset", [(0, 1), (1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("rows,cols", [(21, 64), (21, 777), (21, 4096), (1300, 520)])
def test_strides_alignment_and_guards(b2g, rows, cols, ld_extra, offset, dtype):
    gen = torch.Generator().manual_seed(cols + ld_extra)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, _ = padded(mk(rows, cols), dtype, cols + ld_extra, offset)
    res, _ = padded(mk(rows, cols), dtype, cols + ld_extra, 0)
    w = mk(cols).to(dtype).cuda()
    out, flat = padded(torch.zeros(rows, cols, dtype=torch.float64), dtype, cols + ld_extra + 2,
                       offset)
    before = flat.clone()
    y, total, rstd = b2g.rms_norm(x, w, res, EPS, out=out)
    assert y is out and untouched(flat, out, before)
    check_forward(x, res, w, y, total, rstd)
    # results elsewhere may be added up in another order: the same bounds, not the same bits
    got = b2g.rms_norm_8bit(x, w, res, EPS, with_y=True, keep_total=True)
    check_y8(got[3], *check_forward(x, res, w, *got[:3]))
    assert all(e8.same_bytes(a, b) for a, b in zip(got[4], b2g.quantize_8bit(total)))
    dy, _ = padded(mk(rows, cols), dtype, cols + ld_extra, offset)
    before = flat.clone()
    check_backward(b2g, dy, total, w, rstd, res, out=out)
    assert untouched(flat, out, before)
    kept = e8.make(total, offset=offset, ld=cols + ld_extra, lds=-(-cols // 32) + ld_extra)
    check_backward(b2g, dy, kept, w, rstd, res, out=out)
    assert untouched(flat, out, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(37, 512), (37, 1001), (37, 20000), (1500, 1024)])
def test_in_place(b2g, rows, cols, dtype):
    gen = torch.Generator().manual_seed(cols)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, res, dy, dt = (mk(rows, cols).to(dtype).cuda() for _ in range(4))
    w = mk(cols).to(dtype).cuda()
    y, total, rstd = b2g.rms_norm(x, w, res)
    for k in range(2):
        args = [x.clone(), res.clone()]
        got = b2g.rms_norm(args[0], w, args[1], out=args[k])
        assert all(torch.equal(p, q) for p, q in zip(got, (y, total, rstd)))
    dx, dw = b2g.rms_norm_backward(dy, total, w, rstd, dt)
    for k in range(2):
        args = [dy.clone(), dt.clone()]
        got = b2g.rms_norm_backward(args[0], total, w, rstd, args[1], out=args[k])
        assert got[0] is args[k] and torch.equal(got[0], dx) and torch.equal(got[1], dw)


def test_nonfinite_and_zero_rows(b2g):
    x = torch.randn(6, 300, device="cuda")
    x[1, 7], x[2, 299], x[4] = float("inf"), float("nan"), 0.0
    y, _, rstd, y8, _ = b2g.rms_norm_8bit(x, with_y=True)
    assert not y[4].any() and abs(float(rstd[4]) - EPS ** -0.5) < 1e-3
    assert float(rstd[1]) == 0 and torch.isnan(y[1, 7]) and torch.isnan(y[2]).all()
    v = b2g.dequantize_8bit(*y8)
    assert torch.equal(torch.isnan(v), torch.isnan(y)) and not v[4].any()
    for k in (0, 3, 5):
        assert torch.isfinite(y[k]).all()


def test_no_rows_or_columns(b2g):
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    y, total, rstd = b2g.rms_norm(x, w, x)
    dx, dw = b2g.rms_norm_backward(x, total, w, rstd)
    assert y.shape == dx.shape == (0, 64) and dw.shape == (64,) and not dw.any()
    x = torch.empty(9, 0, device="cuda")
    y, total, rstd = b2g.rms_norm(x)
    assert torch.isnan(rstd).all() and b2g.rms_norm_8bit(x)[3][0].shape == (9, 0)
    dx, dw = b2g.rms_norm_backward(x, total, torch.empty(0, device="cuda"), rstd)
    assert dx.shape == (9, 0) and dw.shape == (0,)


def test_same_bits_every_run(b2g):
    x = torch.randn(3000, 1025, device="cuda")
    w = torch.randn(1025, device="cuda")
    y, total, rstd = b2g.rms_norm(x, w, x)
    first = b2g.rms_norm_backward(y, total, w, rstd, x)
    for _ in range(5):
        assert all(torch.equal(p, q)
                   for p, q in zip(first, b2g.rms_norm_backward(y, total, w, rstd, x)))


def test_gradient_against_differences(b2g):
    """d/dt of sum(dy y) + sum(dtotal total) along x, the residual and the weight, by central
    differences of the forward call itself."""
    torch.manual_seed(3)
    x, res, w, dy, dt = (torch.randn(*s, device="cuda")
                         for s in ((12, 96), (12, 96), (96,), (12, 96), (12, 96)))
    _, total, rstd = b2g.rms_norm(x, w, res)
    dx, dw = b2g.rms_norm_backward(dy, total, w, rstd, dt)
    eps = 2.0 ** -7
    for k, g in enumerate((dx, dw, dx)):
        u = torch.randn_like((x, w, res)[k])

        def loss(t):
            args = [x, w, res]
            args[k] = args[k] + t * u
            y, s, _ = b2g.rms_norm(*args)
            return float((y.double() * dy.double()).sum() + (s.double() * dt.double()).sum())

        diff, trunc = directional(loss, eps)
        y, s, _ = b2g.rms_norm(x, w, res)
        # both ends carry the forward's error (as in check_forward) and that of forming x + t u
        rel = gamma(96) / 2 + 16 * U32
        noise = float((dy.double().abs() * y.abs() + dt.double().abs() * s.abs()).sum()) * rel * 4 / eps
        want = float((g.double() * u.double()).sum())
        assert abs(diff - want) <= trunc + noise, (k, diff, want, trunc, noise)


def test_other_stream_and_graphs(b2g):
    """Another stream; two captured graphs replayed in turn, each with its own workspace."""
    torch.manual_seed(5)
    x, dy = (torch.randn(2000, 1024, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(1024, device="cuda").bfloat16()
    y, total, rstd = b2g.rms_norm(x, w, dy)
    dx, dw = b2g.rms_norm_backward(dy, total, w, rstd, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b2g.rms_norm(x, w, dy, stream=s)
    back = b2g.rms_norm_backward(dy, got[1], w, got[2], x, stream=s)
    eight = b2g.rms_norm_8bit(x, w, dy, with_y=True, keep_total=True, stream=s)
    s.synchronize()
    assert torch.equal(got[0], y) and torch.equal(back[0], dx) and torch.equal(back[1], dw)
    assert torch.equal(eight[0], y)
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f = b2g.rms_norm_8bit(x, w, dy, with_y=True, keep_total=True)
            outs.append((f, b2g.rms_norm_backward(dy, f[4] if k else f[1], w, f[2], x)))
        graphs.append(g)
    for k in (0, 1, 0, 1):
        x.mul_(1.25), dy.mul_(-0.75)
        graphs[k].replay()
        f = b2g.rms_norm_8bit(x, w, dy, with_y=True, keep_total=True)
        want = b2g.rms_norm_backward(dy, f[4] if k else f[1], w, f[2], x)
        torch.cuda.synchronize()
        assert torch.equal(outs[k][0][0], f[0])
        assert all(torch.equal(p, q) for p, q in zip(outs[k][1], want))


def test_rows_past_32_bits_of_offset(b2g):
    flat = torch.zeros(70000, 32768, dtype=BF16, device="cuda")
    x, out = flat[:, :48], flat[:, 64:112]
    x[0], x[-1] = 3.0, -2.0
    y, _, rstd = b2g.rms_norm(x, eps=0.25, out=out)
    want = torch.tensor([9.25, 4.25], dtype=torch.float64).rsqrt()
    close(rstd[[0, -1]], want, want * 1e-6)
    close(y[0], torch.full((48,), 3 * float(want[0])), 3 * 2.0 ** -8)
    close(y[-1], torch.full((48,), -2 * float(want[1])), 2 * 2.0 ** -8)
    assert not y[1:-1].any()
    dx, dw = b2g.rms_norm_backward(x, x, torch.ones(48, device="cuda", dtype=BF16), rstd, out=out)
    assert not dx[1:-1].any() and dx[0].any() and dx[-1].any()
    close(dw, torch.full((48,), float(9 * want[0] + 4 * want[1])), 2.0 ** -8 * 10)


@pytest.mark.parametrize("cols", [2048, 2032, 2047])
@pytest.mark.parametrize("eight", [False, True])
def test_bounded_waits_of_the_rings(b2g, cols, eight):
    """With each group's copies stopped after one row the waits run out, the call returns and
    the status word says so; the next call works again."""
    x = torch.randn(8192, cols, device="cuda").bfloat16()
    w = torch.randn(cols, device="cuda").bfloat16()
    stream = torch.cuda.current_stream().cuda_stream
    y, total, rstd = b2g.rms_norm(x, w, x)
    kept = b2g.quantize_8bit(total) if eight else total
    first = b2g.rms_norm_backward(y, kept, w, rstd, x)
    torch.cuda.synchronize()
    try:
        b2g.b2g_set_wait_limit_ns(2_000_000)
        b2g.b2g_debug_stop_after(1)
        b2g.rms_norm_backward(y, kept, w, rstd, x)
        rc, flags = b2g.b2g_status(stream)
        assert rc == b2g.B2G_ERR_TIMEOUT and flags & 1 and flags & 4
    finally:
        b2g.b2g_debug_stop_after(-1)
        b2g.b2g_set_wait_limit_ns(2_000_000_000)
    again = b2g.rms_norm_backward(y, kept, w, rstd, x)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    assert b2g.b2g_status(stream) == (0, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,ld,offset", [
    (1500, 1001, 1001, 0), (1500, 1001, 1001, 3), (3000, 515, 516, 1), (700, 4099, 4099, 5), (5000, 33, 33, 1),
    (400, 8185, 8185, 2), (1, 777, 777, 7), (3, 5, 5, 1)])
def test_rows_at_one_place_in_their_units(b2g, rows, cols, ld, offset, dtype):
    """All matrices with the same width, stride and offset, off the 16-byte boundaries."""
    gen = torch.Generator().manual_seed(rows + cols)
    mk = lambda: padded(torch.randn(rows, cols, generator=gen, dtype=torch.float64), dtype, ld,  # noqa: E731
                        offset)[0]
    x, dy, dtotal = mk(), mk(), mk()
    w = torch.randn(cols, generator=gen, dtype=torch.float64).to(dtype).cuda()
    out, flat = padded(torch.zeros(rows, cols, dtype=torch.float64), dtype, ld, offset)
    before = flat.clone()
    y, total, rstd = b2g.rms_norm(x, w, out=out)
    assert untouched(flat, out, before)
    check_forward(x, None, w, y, total, rstd)
    check_backward(b2g, dy, x, w, rstd, dtotal, out=out)
    assert untouched(flat, out, before)
    check_backward(b2g, dy, b2g.quantize_8bit(x), w, rstd, None, out=out)
    assert untouched(flat, out, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,offset", [(40, 512, 0), (40, 513, 0), (40, 513, 3), (3, 20001, 1), (700, 96, 1)])
def test_sum_over_the_residual(b2g, rows, cols, offset, dtype):
    """The C call's total may stand where x or the residual was, and y where x was."""
    gen = torch.Generator().manual_seed(cols)
    mk = lambda o: padded(torch.randn(rows, cols, generator=gen, dtype=torch.float64), dtype, cols, o)[0]  # noqa: E731
    x, res = mk(offset), mk(0)
    w = torch.randn(cols, generator=gen, dtype=torch.float64).to(dtype).cuda()
    want = b2g.rms_norm(x, w, res, EPS)
    lib, st = b2g.train_library(), torch.cuda.current_stream().cuda_stream
    code = 0 if dtype is F32 else 1
    for over in range(2):
        args = [x.clone(), res.clone()] if offset == 0 else [mk(offset).copy_(x), mk(0).copy_(res)]
        y = args[0] if over else torch.empty_like(x)
        rstd = torch.empty(rows, device="cuda")
        rc = lib.b2g_rmsnorm(code, rows, cols, args[0].data_ptr(), cols, args[1].data_ptr(), cols, w.data_ptr(),
                             EPS, args[1].data_ptr(), cols, y.data_ptr(), cols, None, 0, None, 0, None, 0, None,
                             0, rstd.data_ptr(), st)
        torch.cuda.synchronize()
        assert rc == 0 and torch.equal(args[1], want[1])
        check_forward(x, res, w, y, args[1], rstd)


def test_scales_that_are_nan(b2g):
    """A NaN scale makes its own row's results NaN, whatever the rows beside it hold."""
    for cols in (96, 1000, 1001):
        x = torch.randn(1500, cols, device="cuda")
        kept = b2g.quantize_8bit(x)
        kept[1].view(torch.uint8)[7, 1] = 255
        rstd = torch.ones(1500, device="cuda")
        dx, _ = b2g.rms_norm_backward(x, kept, None, rstd)
        assert torch.isnan(dx[7]).all() and torch.isfinite(dx[:7]).all() and torch.isfinite(dx[8:]).all()


@pytest.mark.parametrize("rows,cols", [(16, 4096), (9, 777)])
def test_few_rows_captured_and_on_another_stream(b2g, rows, cols):
    x, dy, dtotal = (torch.randn(rows, cols, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(cols, device="cuda").bfloat16()
    _, total, rstd = b2g.rms_norm(x, w)
    want = b2g.rms_norm_backward(dy, total, w, rstd, dtotal)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = b2g.rms_norm_backward(dy, total, w, rstd, dtotal, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [b2g.rms_norm_backward(dy, total, w, rstd, dtotal) for _ in range(3)]
    for _ in range(3):
        dy.mul_(1.25)
        g.replay()
        want = b2g.rms_norm_backward(dy, total, w, rstd, dtotal)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))
