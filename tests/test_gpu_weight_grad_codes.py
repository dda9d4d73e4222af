"""The weight gradient that converts x from its codes within the product's kernel, where each
CTA of a pair reads tiles that warps of the other one wrote: the same bits every time, over
many k tiles and many tiles, and beside other work on the GPU."""
import pytest
import torch

import eightbit_helpers as e8
from gpu_helpers import env
from test_gpu_weight_grad import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


# few tokens on many tiles, many tokens on few tiles, and between; halves of tiles, pieces of
# tiles, ends of 16 columns and of 64 tokens
SIZES = [(300, 512, 256), (64, 4096, 4096), (130, 2048, 4096), (1000, 130, 4000), (5000, 128, 1008),
         (4096, 512, 520), (5844, 128, 6944), (16384, 128, 1024), (2048, 1024, 1024), (20001, 64, 200)]


@pytest.mark.parametrize("tokens,outs,width", SIZES)
def test_same_bits_every_time(b2g, tokens, outs, width):
    torch.manual_seed(tokens + outs + width)
    dy = torch.randn(tokens, outs, device="cuda").to(BF16)
    kept = b2g.quantize_8bit(torch.randn(tokens, width, device="cuda"))
    first = b2g.linear_weight_grad_8bit(dy, *kept)
    check(first, dy, e8.values(*kept))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(100):
        if i % 4 == 0:  # norms and conversions of the side stream share the SMs' caches and HBM
            b2g.quantize_8bit(dy, stream=side)
        assert torch.equal(first, b2g.linear_weight_grad_8bit(dy, *kept)), i
    side.synchronize()
