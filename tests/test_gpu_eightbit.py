"""Rows to their 8-bit form and back on the GPU: the same bytes and values as the
definition in 64 bits."""
import pytest
import torch

import eightbit_helpers as e8
from gpu_helpers import env
from train_helpers import padded, untouched

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def spread(rows, cols, seed, range_=6.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    return x * torch.exp(range_ * torch.randn(rows, cols, generator=g, dtype=torch.float64))


SHAPES = [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (1, 4096), (19, 64), (33, 1000), (40, 1025),
          (7, 8192), (3, 20001), (700, 96), (2000, 48), (1217, 264), (300, 777)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_and_back(b2g, rows, cols, dtype):
    x = spread(rows, cols, rows * 7 + cols).to(dtype).cuda()
    codes, scales = b2g.quantize_8bit(x)
    want = e8.encode(x)
    assert codes.shape == x.shape and codes.stride(0) % 16 == 0
    assert e8.same_bytes(scales, want[1]) and e8.same_bytes(codes, want[0])
    v = e8.values(codes, scales)
    for dt in (F32, BF16):
        # 4 significant bits and a scale of 2^-110 or more: exact in both types
        assert torch.equal(b2g.dequantize_8bit(codes, scales, dt).double().cpu(), v)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset,extra", [(0, 0), (1, 0), (0, 3), (8, 8), (5, 11)])
@pytest.mark.parametrize("cols", [64, 200, 777])
def test_strides_and_guards(b2g, cols, offset, extra, dtype):
    x, _ = padded(spread(21, cols, cols), dtype, cols + extra, offset)
    codes, scales = b2g.quantize_8bit(x)
    want = e8.encode(x)
    assert e8.same_bytes(codes, want[0]) and e8.same_bytes(scales, want[1])
    given = e8.make(x, offset=offset, ld=cols + extra + 1, lds=-(-cols // 32) + extra)
    out, flat = padded(torch.zeros(21, cols, dtype=torch.float64), dtype, cols + extra + 2, offset)
    before = flat.clone()
    assert b2g.dequantize_8bit(*given, out=out) is out
    assert untouched(flat, out, before)
    assert torch.equal(out.double().cpu(), e8.values(*given))


def test_borders_of_the_scale(b2g):
    """Blocks whose largest value is 448 powers of two, its neighbours, zero, tiny, huge."""
    top = [448.0 * 2.0 ** k for k in (-125, -119, -118, -100, -1, 0, 1, 100, 119)]
    f = torch.tensor(top, dtype=F32)
    rows = torch.cat([f, torch.nextafter(f, torch.zeros_like(f)), torch.nextafter(f, f * 2),
                      torch.tensor([0.0, 1e-45, 2.0 ** -126, 3e38, 2.0 ** -149 * 5])])
    x = torch.zeros(rows.numel(), 40)
    x[:, 3] = rows
    x[:, 11] = -rows / 3
    x[:, 35] = rows / 7  # another block
    for dt in (F32, BF16):
        y = x.to(dt).cuda()
        codes, scales = b2g.quantize_8bit(y)
        want = e8.encode(y)
        assert e8.same_bytes(scales, want[1]) and e8.same_bytes(codes, want[0])


@pytest.mark.parametrize("cols", [64, 45])
def test_infinities_and_nan(b2g, cols):
    """They become NaN; the others of their block keep the scale of the finite values."""
    for dt in (F32, BF16):
        x = spread(9, cols, 3, 1.0).to(dt)
        x[0, 1], x[1, 40], x[2, 2], x[2, 3] = float("inf"), float("-inf"), float("nan"), float("inf")
        x[3] = float("nan")
        x[4, :32] = float("inf")
        x[5, 31] = float("nan")
        x = x.cuda()
        codes, scales = b2g.quantize_8bit(x)
        want = e8.encode(x)
        assert e8.same_bytes(scales, want[1])
        got, expect = e8.values(codes, scales), e8.values(*want)
        assert torch.equal(torch.isnan(got), ~torch.isfinite(x.cpu()))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(expect))


def test_every_code_and_scale(b2g):
    """256 codes at 256 scales: rounded once to either type."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8).contiguous().cuda()
    q, s = codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    v = e8.values(q, s)
    for dt in (F32, BF16):
        got = b2g.dequantize_8bit(q, s, dt).cpu()
        want = v.float().to(dt)  # 4 significant bits: FP32 holds every one below its largest
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def test_no_rows_or_columns(b2g):
    for shape in ((0, 64), (5, 0), (0, 0)):
        codes, scales = b2g.quantize_8bit(torch.empty(*shape, device="cuda"))
        assert codes.shape == shape and scales.shape == (shape[0], -(-shape[1] // 32))
        assert b2g.dequantize_8bit(codes, scales).shape == shape


def test_other_stream_and_graph(b2g):
    x = torch.randn(513, 1032, device="cuda")
    want = e8.encode(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = b2g.quantize_8bit(x, stream=s)
    back = b2g.dequantize_8bit(codes, scales, F32, stream=s)
    s.synchronize()
    assert e8.same_bytes(codes, want[0]) and torch.equal(back.double().cpu(), e8.values(*want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        codes, scales = b2g.quantize_8bit(x)
        back = b2g.dequantize_8bit(codes, scales, F32)
    x.mul_(-3.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(back.double().cpu(), e8.values(*e8.encode(x)))


def test_rows_past_32_bits_of_offset(b2g):
    """Rows that begin more than 2^31 elements after the first one."""
    flat = torch.zeros(70000 * 32768, dtype=BF16, device="cuda")
    x = flat.view(70000, 32768)[:, :40]
    x[0], x[-1] = 3.0, -5.0
    codes, scales = b2g.quantize_8bit(x)
    back = b2g.dequantize_8bit(codes, scales, BF16, out=flat.view(70000, 32768)[:, 64:104])
    assert torch.equal(back, x) and int((back != 0).sum()) == 80
