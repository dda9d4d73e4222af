"""The weight gradient from inputs kept in 8 bits against the product in 64 bits."""
import pytest
import torch

import eightbit_helpers as e8
from gpu_helpers import env
from train_helpers import TINY, U, close, directional, padded, untouched

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def steps(tokens):
    """Roundings that a result's sum meets, in units of 2^-23 of the sum of absolute values
    (an addition that truncates): one for each 16 tokens and three for FP32's pieces; 8 for
    the alignment of the 16 products of a step, 2^-24 of the largest each; one for each
    slice of the tokens and 16 to spare."""
    return 3 * (tokens / 16 + 1) + 8 + 76 + 16


def check(dw, dy, x, old=None):
    D, X = dy.double(), x.double().to(dy.device)
    want = D.t() @ X + (0 if old is None else old.double())
    size = D.abs().t() @ X.abs() + (0 if old is None else old.double().abs())
    close(dw, want, steps(len(dy)) * 2.0 ** -23 * size + U[dy.dtype] * want.abs() * (1 + 1e-4) + TINY, "dw")


def operands(tokens, outs, width, dtype, seed=0, **kw):
    g = torch.Generator().manual_seed(seed + tokens + 3 * outs + 7 * width)
    mk = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    dy = mk(tokens, outs).to(dtype).cuda()
    x = mk(tokens, width) * torch.exp(2 * mk(tokens, width))
    return dy, e8.make(x, **kw)


SHAPES = [(1, 1, 1), (3, 5, 33), (64, 64, 64), (65, 130, 257), (300, 512, 256), (1000, 1025, 777),
          (17, 300, 31), (2000, 96, 4000), (5000, 40, 70), (16, 4096, 4096), (128, 256, 256),
          (129, 255, 128), (4096, 512, 520), (700, 1200, 264), (40000, 24, 72), (1, 8, 16), (63, 72, 48), (1000, 264, 784),
          (5000, 128, 1008), (70, 4096, 4096), (3000, 64, 6944), (20000, 64, 64), (40000, 40, 144)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,outs,width", SHAPES)
def test_against_64_bits(b2g, tokens, outs, width, dtype):
    dy, kept = operands(tokens, outs, width, dtype)
    check(b2g.linear_weight_grad_8bit(dy, *kept), dy, e8.values(*kept))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,outs,width", [(70, 96, 200), (1000, 130, 77), (900, 520, 776)])
@pytest.mark.parametrize("offset,extra", [(1, 0), (0, 3), (8, 8), (16, 16)])
def test_strides_accumulate_and_guards(b2g, tokens, outs, width, offset, extra, dtype):
    host = torch.randn(tokens, outs, dtype=torch.float64)
    dy, _ = padded(host, dtype, outs + extra, offset)
    _, kept = operands(tokens, outs, width, dtype, offset=offset, ld=width + extra,
                       lds=-(-width // 32) + extra)
    x = e8.values(*kept)
    old = torch.randn(outs, width, dtype=torch.float64)
    for accumulate in (False, True):
        out, flat = padded(old, dtype, width + extra, offset)
        before, was = flat.clone(), out.clone()
        assert b2g.linear_weight_grad_8bit(dy, *kept, dw=out, accumulate=accumulate) is out
        assert untouched(flat, out, before)
        check(out, dy, x, was if accumulate else None)


@pytest.mark.parametrize("lds", [0, 3])
@pytest.mark.parametrize("tokens,outs,width", [
    (70, 96, 200), (900, 520, 776), (900, 77, 1000), (1, 8, 8), (2000, 100, 136), (129, 1000, 72), (64, 300, 1000),
    (65, 256, 264), (3000, 64, 520), (333, 264, 24), (1024, 2048, 2048), (2500, 600, 640)])
def test_aligned_rows_in_larger_buffers(b2g, tokens, outs, width, lds):
    """All rows on 16-byte boundaries, widths that end inside 16 and 32 columns; NaN codes and
    scales behind x's rows, and nothing written behind dw's."""
    dy, kept = operands(tokens, outs, width, BF16, seed=lds, lds=-(-width // 32) + lds,
                        ld=-(-width // 16) * 16 + 16)
    dy, _ = padded(dy.cpu().double(), BF16, -(-outs // 8) * 8 + 8)
    out, flat = padded(torch.zeros(outs, width, dtype=torch.float64), BF16, width + 8)
    before = flat.clone()
    assert b2g.linear_weight_grad_8bit(dy, *kept, dw=out) is out
    assert untouched(flat, out, before)
    check(out, dy, e8.values(*kept))
    odd, _ = padded(dy.cpu().double(), BF16, outs + 1, 3)
    check(b2g.linear_weight_grad_8bit(odd, *kept), dy, e8.values(*kept))
    # the same values in rows off the boundaries take the other way
    _, other = operands(tokens, outs, width, BF16, seed=lds, offset=1, ld=width + 1)
    check(b2g.linear_weight_grad_8bit(dy, *other), dy, e8.values(*kept))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld", [256, 257])
def test_every_code_and_scale(b2g, ld, dtype):
    """dy = the identity returns x's values: exactly, each is one BF16 number.  Scales from 2^-110
    up to the largest whose products with 448 BF16 holds."""
    r, c = torch.arange(256)[:, None], torch.arange(256)[None]
    codes = ((r + c) % 256).to(torch.uint8)
    codes[codes & 127 == 127] = 0
    scales = (17 + (8 * r + torch.arange(8)[None]) % 230).to(torch.uint8)
    flat = torch.zeros(256, ld, dtype=torch.uint8, device="cuda")
    flat[:, :256] = codes
    kept = flat.view(torch.float8_e4m3fn)[:, :256], scales.cuda().view(torch.float8_e8m0fnu)
    dw = b2g.linear_weight_grad_8bit(torch.eye(256, dtype=dtype, device="cuda"), *kept)
    assert torch.equal(dw.cpu().double(), e8.values(*kept))
    # NaN stays in its column, a NaN scale in its 32
    flat[5, 40], flat[255, 200] = 127, 255
    kept[1].view(torch.uint8)[7, 3] = 255
    dw = b2g.linear_weight_grad_8bit(torch.eye(256, dtype=dtype, device="cuda"), *kept)
    lost = torch.zeros(256, dtype=torch.bool, device="cuda")
    lost[40] = lost[200] = lost[96:128] = True
    assert torch.isnan(dw[:, lost]).all() and torch.isfinite(dw[:, ~lost]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_tokens(b2g, dtype):
    dy = torch.empty(0, 40, dtype=dtype, device="cuda")
    kept = b2g.quantize_8bit(torch.empty(0, 72, dtype=dtype, device="cuda"))
    assert not b2g.linear_weight_grad_8bit(dy, *kept).any()
    old = torch.ones(40, 72, dtype=dtype, device="cuda")
    b2g.linear_weight_grad_8bit(dy, *kept, dw=old, accumulate=True)
    assert (old == 1).all()
    dy = torch.ones(5, 0, dtype=dtype, device="cuda")
    kept = b2g.quantize_8bit(torch.ones(5, 72, dtype=dtype, device="cuda"))
    assert b2g.linear_weight_grad_8bit(dy, *kept).shape == (0, 72)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nonfinite_columns(b2g, dtype):
    """A NaN that was kept reaches its column of dw and no other."""
    dy, kept = operands(300, 140, 520, dtype)
    bytes_ = kept[0].view(torch.uint8)
    bytes_[299, 519] = 0x7f
    dw = b2g.linear_weight_grad_8bit(dy, *kept)
    assert torch.isnan(dw[:, 519]).all() and torch.isfinite(dw[:, :519]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_and_small_values(b2g, dtype):
    """dy over FP32's range of exponents, and scales at both ends of theirs."""
    dy, kept = operands(200, 64, 96, dtype)
    x = torch.randn(200, 96, dtype=torch.float64)
    for a, b in ((2.0 ** -100, 2.0 ** 90), (2.0 ** 100, 2.0 ** -100), (2.0 ** -60, 2.0 ** -60)):
        small = (dy.double() * a).to(dtype)
        k = e8.make(x * b)
        check(b2g.linear_weight_grad_8bit(small, *k), small, e8.values(*k))


def test_terms_of_one_sign(b2g):
    """Many tokens whose terms do not cancel: truncated sums would show as a bias."""
    for dtype, tokens in ((F32, 70000), (BF16, 300000)):
        dy = (torch.rand(tokens, 16, device="cuda") + 0.5).to(dtype)
        x = torch.rand(tokens, 32, device="cuda") + 0.5
        kept = b2g.quantize_8bit(x)
        dw = b2g.linear_weight_grad_8bit(dy, *kept)
        want = dy.double().t() @ e8.values(*kept).cuda()
        # FP32: at most 256 tokens add up with truncation, 48 steps of three pieces and 8 units
        # for their products' alignment, 2^-23 each; those sums with rounding, 2^-24 each.
        # BF16: the result's rounding, and 2^-12 of truncation.
        rel = 56 * 2.0 ** -23 + tokens / 256 * 2.0 ** -24 if dtype is F32 else 2.0 ** -8 + 2.0 ** -12
        close(dw, want, want * rel, "dw")


def test_same_bits_every_run(b2g):
    dy, kept = operands(3000, 300, 500, BF16)
    first = b2g.linear_weight_grad_8bit(dy, *kept)
    for _ in range(5):
        assert torch.equal(first, b2g.linear_weight_grad_8bit(dy, *kept))


def test_gradient_against_differences(b2g):
    """dw against central differences of sum(dy * (x w^T)), linear in w: by its truncation
    alone."""
    dy, kept = operands(40, 24, 56, F32)
    x = e8.values(*kept)
    dw = b2g.linear_weight_grad_8bit(dy, *kept).double().cpu()
    torch.manual_seed(1)
    w, u = (torch.randn(24, 56, dtype=torch.float64) for _ in range(2))
    diff, trunc = directional(lambda t: float((dy.double().cpu() * (x @ (w + t * u).t())).sum()), 0.5)
    size = dy.double().abs().cpu().t() @ x.abs()
    assert abs(diff - float((dw * u).sum())) <= trunc + float(
        (size * u.abs()).sum()) * steps(40) * 2.0 ** -23


def test_other_stream_and_graphs(b2g):
    for dtype in (F32, BF16):
        dy, kept = operands(700, 264, 520, dtype)
        want = b2g.linear_weight_grad_8bit(dy, *kept)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = b2g.linear_weight_grad_8bit(dy, *kept, stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(b2g.linear_weight_grad_8bit(dy, *kept))
            graphs.append(g)
        for k in (0, 1, 0):
            dy.mul_(1.5)
            graphs[k].replay()
            want = b2g.linear_weight_grad_8bit(dy, *kept)
            torch.cuda.synchronize()
            assert torch.equal(outs[k], want)


@pytest.mark.parametrize("tokens,outs,width", [(300, 512, 256), (1000, 128, 4096), (64, 100, 255)])
def test_two_streams_at_once(b2g, tokens, outs, width):
    """Calls that run side by side, one writing over its own result and one adding to it."""
    dy, kept = operands(tokens, outs, width, BF16)
    want = b2g.linear_weight_grad_8bit(dy, *kept)
    twice = b2g.linear_weight_grad_8bit(dy, *kept, dw=want.clone(), accumulate=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs8 = [[], []]
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                dw = b2g.linear_weight_grad_8bit(dy, *kept)
                if k:
                    assert b2g.linear_weight_grad_8bit(dy, *kept, dw=dw, accumulate=True) is dw
                outs8[k].append(dw)
    torch.cuda.synchronize()
    assert all(torch.equal(dw, want) for dw in outs8[0])
    assert all(torch.equal(dw, twice) for dw in outs8[1])


def test_rows_past_32_bits_of_offset(b2g):
    flat = torch.zeros(70000, 32768, dtype=BF16, device="cuda")
    dy = flat[:, :40]
    dy[0], dy[-1] = 3.0, -5.0
    x = torch.ones(70000, 48, dtype=BF16, device="cuda")
    dw = b2g.linear_weight_grad_8bit(dy, *b2g.quantize_8bit(x))
    assert (dw == -2).all()


def test_codes_past_32_bits_of_offset(b2g):
    flat = torch.zeros(20000, 1 << 18, dtype=torch.uint8, device="cuda")
    scales = torch.full((20000, 1 << 17), 127, dtype=torch.uint8, device="cuda")
    flat[0, :64], flat[-1, :64] = 0x38, 0xC0  # 1 and -2
    scales[-1, :2] = 129
    dw = b2g.linear_weight_grad_8bit(torch.ones(20000, 40, dtype=BF16, device="cuda"),
                                     flat.view(torch.float8_e4m3fn)[:, :64],
                                     scales.view(torch.float8_e8m0fnu)[:, :2])
    assert (dw == 1 - 8).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bounded_waits(b2g, dtype):
    """With the copies stopped the waits run out, the call returns and the status word says
    so; the next call works again."""
    dy, kept = operands(2000, 600, 520, dtype)
    stream = torch.cuda.current_stream().cuda_stream
    first = b2g.linear_weight_grad_8bit(dy, *kept)
    torch.cuda.synchronize()
    try:
        b2g.b2g_set_wait_limit_ns(2_000_000)
        b2g.b2g_debug_stop_after(2)
        b2g.linear_weight_grad_8bit(dy, *kept)
        rc, flags = b2g.b2g_status(stream)
        assert rc == b2g.B2G_ERR_TIMEOUT and flags & 1 and flags & 8
    finally:
        b2g.b2g_debug_stop_after(-1)
        b2g.b2g_set_wait_limit_ns(2_000_000_000)
    assert torch.equal(first, b2g.linear_weight_grad_8bit(dy, *kept))
    assert b2g.b2g_status(stream) == (0, 0)
