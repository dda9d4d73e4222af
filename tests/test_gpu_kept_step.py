"""RMS norms, 8-bit activations, the products and the cross entropy together:
examples/kept_step.py against the same steps in 64 bits."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

import eightbit_helpers as e8

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "kept_step", os.path.join(ROOT, "examples", "kept_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm_gradient(dy, t, w, rstd, past):
    """(dx, dweight) of the norm at rows t, by its formula."""
    xh, g = t * rstd[:, None], dy * w
    return rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True)) + past, (dy * xh).sum(0)


def reference(p, ids, target, eps, kept=None):
    """Mean loss and gradients in 64 bits; `kept`: the values of the 8-bit forms (x, y, t),
    which the backward formulas read in place of the exact rows."""
    q = {k: v.double() for k, v in p.items()}
    x = q["embed"][ids]
    r1 = (x.square().mean(1) + eps).rsqrt()
    y = x * r1[:, None] * q["norm1"]
    t = x + y @ q["layer"].t()
    r2 = (t.square().mean(1) + eps).rsqrt()
    h = (t * r2[:, None] * q["norm2"]).requires_grad_()
    head = q["embed"].clone().requires_grad_()
    loss = F.cross_entropy(h @ head.t(), target)
    loss.backward()
    kx, ky, kt = kept or (x, y, t)
    dt, dnorm2 = norm_gradient(h.grad, kt, q["norm2"], r2, 0)
    dlayer = dt.t() @ ky
    dx, dnorm1 = norm_gradient(dt @ q["layer"], kx, q["norm1"], r1, dt)
    dembed = head.grad.index_add(0, ids, dx)
    return float(loss.detach()), {"embed": dembed, "layer": dlayer, "norm1": dnorm1, "norm2": dnorm2}, (x, y, t)


@pytest.mark.parametrize("vocab,width,tokens", [(50, 16, 7), (1000, 128, 300), (1001, 129, 301), (130, 64, 1000)])
def test_gradients(vocab, width, tokens):
    ex = example()
    p = ex.parameters(vocab, width, seed=3)
    ids, target = ex.batch(vocab, tokens, seed=4)
    loss, kept = ex.forward(p, ids, target)
    check(ex, p, ids, target, loss, kept, ex.backward(p, ids, target, kept))


def check(ex, p, ids, target, loss, kept, grads):
    (vocab, width), tokens = p["embed"].shape, ids.numel()
    held = [e8.values(*kept[k]).cuda() for k in ("x8", "y8", "t8")]
    want_loss, want, exact = reference(p, ids, target, ex.EPS, held)
    # each kept value is its row's, once rounded to 4 bits: 2^-4 of it, or 2^-10 of a scale that
    # is at most 2 / 448 of the block's largest, with FP32's errors of the row itself
    for v, e in zip(held, exact):
        top = F.pad(e.abs(), (0, -width % 32)).view(tokens, -1, 32).amax(2).repeat_interleave(32, 1)[:, :width]
        assert ((v - e).abs() <= torch.maximum(2.0 ** -4 * e.abs(), 2.0 ** -17 * top) + 1e-5 * top).all()
    # About ten operators in a row, each of whose sums of at most L terms is within L 2^-24 of
    # the sum of absolute values; a factor of 4 for sums that cancel.  (In norm over a whole
    # tensor: the bound is far from what is expected.)
    bound = 4 * 10 * max(vocab, width, tokens) * 2.0 ** -24
    assert abs(float(loss.mean()) - want_loss) <= bound * abs(want_loss)
    for name, g in want.items():
        err = float((grads[name].double() - g).norm())
        assert err <= bound * float(g.norm()), (name, err, float(g.norm()))


def test_gradients_against_exact_ones():
    """What 8 bits cost the gradients: the formulas read rows that are off by at most 2^-4 of
    each value (a uniform error of that size has a third of its square on average), twice in
    the norms'."""
    ex = example()
    p = ex.parameters(500, 128, seed=5)
    ids, target = ex.batch(500, 400, seed=6)
    _, kept = ex.forward(p, ids, target)
    grads = ex.backward(p, ids, target, kept)
    _, want, _ = reference(p, ids, target, ex.EPS)
    for name, g in want.items():
        assert float((grads[name].double() - g).norm()) <= 2 * 2.0 ** -4 * float(g.norm()), name


def test_it_runs():
    losses = example().train(vocab=200, width=64, tokens=1024, steps=5)
    assert len(losses) == 5 and all(0 < v < 20 for v in losses)


def test_two_runs_same_bits():
    ex = example()
    a, b = (ex.train(vocab=130, width=48, tokens=257, steps=5) for _ in range(2))
    assert a == b


def test_captured_step():
    """The whole step in one graph, replayed on other tokens."""
    ex = example()
    p = ex.parameters(300, 96, seed=1)
    ids, target = ex.batch(300, 200, seed=2)
    ex.backward(p, ids, target, ex.forward(p, ids, target)[1])  # libraries loaded, kernels set up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, kept = ex.forward(p, ids, target)
        grads = ex.backward(p, ids, target, kept)
    for seed in (3, 4):
        new_ids, new_target = ex.batch(300, 200, seed=seed)
        ids.copy_(new_ids), target.copy_(new_target)
        g.replay()
        torch.cuda.synchronize()
        check(ex, p, new_ids, new_target, loss, kept, grads)
