"""All 24 bits of FP32 gradients in the weight gradient, and where they end."""
import pytest
import torch

import eightbit_helpers as e8
from gpu_helpers import env
from train_helpers import U, close

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def signed(g, *shape):
    return torch.randint(0, 2, shape, generator=g).double() * 2 - 1


def one_token_each(tokens, outs, width, seed, low, high, shift):
    """dy whose columns have one nonzero token each, of random 24 bits and an exponent of
    [low, high), and x of powers of two from 2^shift to 2^(shift + 7): every element of dw is one
    product, which FP32 holds."""
    g = torch.Generator().manual_seed(seed)
    top = torch.randint(1 << 23, 1 << 24, (outs,), generator=g).double() * 2.0 ** -23  # [1, 2)
    e = torch.randint(low, high, (outs,), generator=g).double()
    at = torch.randint(0, tokens, (outs,), generator=g)
    dy = torch.zeros(tokens, outs, dtype=torch.float64)
    dy[at, torch.arange(outs)] = top * torch.exp2(e) * signed(g, outs)
    x = torch.exp2(torch.randint(0, 8, (tokens, width), generator=g).double() + shift) * signed(g, tokens, width)
    return dy, x


SIZES = [(1, 3, 5), (64, 64, 64), (65, 130, 257), (300, 512, 256), (17, 300, 31), (1000, 1025, 777),
         (3000, 64, 6944), (600, 2575, 1660), (20000, 40, 72)]


@pytest.mark.parametrize("low,high,shift", [(-20, 20, 0), (-110, -100, 60), (90, 127, -100), (-110, 127, -7)])
@pytest.mark.parametrize("tokens,outs,width", SIZES)
def test_every_bit_of_fp32_gradients(b2g, tokens, outs, width, low, high, shift):
    """Three BF16 pieces hold 24 bits from 2^-110 on: the last one's smallest is 2^-133."""
    dy, x = one_token_each(tokens, outs, width, tokens + outs, low, high, shift)
    kept = b2g.quantize_8bit(x.float().cuda())
    assert torch.equal(e8.values(*kept), x)
    want = dy.t() @ x  # one product an element: exact
    keep = torch.isfinite(want.float()) & ((want == 0) | (want.abs() >= 2.0 ** -126))
    dw = b2g.linear_weight_grad_8bit(dy.float().cuda(), *kept)
    assert torch.equal(dw.cpu().double()[keep], want[keep])
    if high < 100:  # added: one rounding of the sum
        old = torch.randn(outs, width, generator=torch.Generator().manual_seed(1)) * 2.0 ** min(low + shift + 20, 100)
        dw = b2g.linear_weight_grad_8bit(dy.float().cuda(), *kept, dw=old.cuda(), accumulate=True)
        assert torch.equal(dw.cpu()[keep], (old + want.float())[keep])


def test_gradients_below_that(b2g):
    """The pieces end at 2^-133: what is left of a smaller dy is off by 2^-134 at most."""
    dy, x = one_token_each(300, 200, 96, 1, -126, -110, 70)
    kept = b2g.quantize_8bit(x.float().cuda())
    want = dy.t() @ x
    dw = b2g.linear_weight_grad_8bit(dy.float().cuda(), *kept)
    big = (dy != 0).double().t() @ x.abs()  # the one |x| of each element
    close(dw, want, 2.0 ** -134 * big + U[F32] * want.abs(), "dw")


def test_many_small_gradients(b2g):
    """The same in sums of 64 products."""
    g = torch.Generator().manual_seed(2)
    dy = (torch.randn(64, 130, generator=g, dtype=torch.float64) * 2.0 ** -120).float()
    kept = b2g.quantize_8bit((torch.randn(64, 264, generator=g) * 2.0 ** 80).cuda())
    x = e8.values(*kept)
    dw = b2g.linear_weight_grad_8bit(dy.cuda(), *kept)
    size = dy.double().abs().t() @ x.abs()
    # four steps of three pieces, truncated, and 8 units for the alignment of their products
    close(dw, dy.double().t() @ x, 20 * 2.0 ** -23 * size + 2.0 ** -134 * x.abs().sum(0), "dw")
