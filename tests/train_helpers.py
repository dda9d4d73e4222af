"""Shared helpers of the training-operator tests: operands with padding,
guard bands and any alignment, and elementwise checks against 64-bit results.

Rounding: U is half a unit in the last place of each type relative to the value,
so a result rounded once from an exact value v is within U * |v| of it.
"""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-37  # values whose rounding is absolute (subnormals)


def padded(host, dtype, ld=None, offset=0, guard=3):
    """`host` (2-D, float64) as a CUDA matrix of `dtype` with row stride ld whose
    first element stands `offset` elements past a 16-byte boundary; the padding
    and `guard` rows below hold NaN.  Returns (view, whole buffer)."""
    r, c = host.shape
    ld = max(ld or c, 1)
    flat = torch.full((offset + (r + guard) * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    view = torch.as_strided(flat, (r, c), (ld, 1), offset)
    view.copy_(host.to(dtype))
    return view, flat


def untouched(flat, view, before):
    """True when every element of the buffer outside the view kept its bits."""
    mask = torch.ones(flat.shape, dtype=torch.bool, device=flat.device)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    bits = torch.int32 if flat.dtype is torch.float32 else torch.int16
    return bool(torch.equal(flat.view(bits)[mask], before.view(bits)[mask]))


def close(got, want, bound, what=""):
    """Every element within its bound of the 64-bit value; NaN and infinities
    where, and only where, the reference has them."""
    got, want = got.double().cpu(), want.double().cpu()
    bound = torch.as_tensor(bound, dtype=torch.float64).cpu().expand_as(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    err = (got - want).abs()[fine]
    over = err > bound[fine]
    if over.any():
        worst = (err / bound[fine].clamp(min=1e-300)).max()
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside the bound, "
                             f"the worst {float(worst):.3g} times")
    return float((err / bound[fine].clamp(min=1e-300)).max()) if err.numel() else 0.0


def directional(loss, eps):
    """The central difference of loss(t) at 0 and a bound on its truncation.

    D(e) = f' + c e^2 + O(e^4), so D(2e) - D(e) is three times the error of D(e);
    the whole difference is allowed, for the higher terms."""
    d1 = (loss(eps) - loss(-eps)) / (2 * eps)
    d2 = (loss(2 * eps) - loss(-2 * eps)) / (4 * eps)
    return d1, abs(d2 - d1)
