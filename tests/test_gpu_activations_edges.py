"""RMS norm and 8-bit activations: calls that the documentation allows and that come up
rarely.  Results given for no elements at all."""
import pytest
import torch

from gpu_helpers import env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_given_results_without_elements(b2g, shape, residual):
    """Empty tensors have one address, and share nothing."""
    x, out = (torch.empty(*shape, device="cuda") for _ in range(2))
    res = torch.empty(*shape, device="cuda") if residual else None
    y, total, rstd = b2g.rms_norm(x, residual=res, out=out)
    assert y is out and total.shape == shape and rstd.shape == shape[:1]
    dx, dw = b2g.rms_norm_backward(x, total, torch.ones(shape[1], device="cuda"), rstd, out=out)
    assert dx is out and dw.shape == shape[1:] and not dw.any()
    kept = b2g.quantize_8bit(x)
    assert b2g.dequantize_8bit(*kept, out=out) is out
    dw = torch.empty(shape[1], shape[1], device="cuda")
    assert b2g.linear_weight_grad_8bit(x, *kept, dw=dw) is dw and not dw.any()
