"""The head's gradient written between other data: the columns beside it keep their bits."""
import pytest
import torch

from gpu_helpers import env
from train_helpers import untouched

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [130, 1000])
@pytest.mark.parametrize("width", [73, 77, 79, 80])
def test_columns_beside_the_gradient(width, tokens, accumulate, dtype):
    b2g = env()[1]
    torch.manual_seed(width + tokens)
    h, head = (torch.randn(n, width, device="cuda").to(dtype) for n in (tokens, 300))
    target = torch.randint(0, 300, (tokens,), device="cuda")
    each = torch.full((tokens,), 1.0 / tokens, device="cuda")
    _, lse = b2g.linear_cross_entropy(h, head, target)
    want = b2g.linear_cross_entropy_backward(h, head, target, lse, each)[1]
    flat = torch.full((303 * 80,), float("nan"), device="cuda", dtype=dtype)
    out = flat[:300 * 80].view(300, 80)[:, :width]  # rows on 16-byte boundaries, the width not
    out.fill_(0.0)
    before = flat.clone()
    b2g.linear_cross_entropy_backward(h, head, target, lse, each, dw=out, accumulate=accumulate)
    assert untouched(flat, out, before) and torch.equal(out, want)
