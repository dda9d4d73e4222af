"""The operators and the SGEMM together: examples/train_step.py against the same
model in 64 bits."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(p, ids, target, eps):
    """Mean loss and gradients of the model by differentiation in 64 bits."""
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    d = (p["layer"].shape[0],)
    x = F.embedding(ids, q["embed"])
    y = x + F.layer_norm(x, d, q["norm1.weight"], q["norm1.bias"], eps) @ q["layer"]
    h = F.layer_norm(y, d, q["norm2.weight"], q["norm2.bias"], eps)
    loss = F.cross_entropy(h @ q["embed"].T, target)
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("vocab,width,tokens,max_norm", [
    (50, 16, 7, 1e9), (1000, 128, 300, 1e9), (1001, 129, 301, 1e9), (130, 64, 40, 0.25)])
def test_gradients(vocab, width, tokens, max_norm):
    ex = example()
    p = ex.parameters(vocab, width, seed=3)
    ids, target = ex.batch(vocab, tokens, seed=4)
    loss, grads, norm = ex.step(p, ids, target, max_norm)
    want_loss, want = reference(p, ids, target, ex.EPS)
    # About ten operators in a row, each of whose sums of at most L terms is within
    # L 2^-24 of the sum of absolute values; a factor of 4 for sums that cancel.
    # (In norm over a whole tensor: the bound is far from what is expected.)
    bound = 4 * 10 * max(vocab, width, tokens) * 2.0 ** -24
    assert abs(float(loss) - want_loss) <= bound * abs(want_loss)
    want_norm = float(torch.stack([g.norm() for g in want.values()]).norm())
    assert abs(float(norm) - want_norm) <= bound * want_norm
    scale = min(1.0, max_norm / (want_norm + 1e-6))
    for name, g in want.items():
        err = float((grads[name].double() - scale * g).norm())
        assert err <= bound * scale * float(g.norm()), (name, err, float(g.norm()))


def test_loss_falls():
    """From about log(vocab) to less than half of it."""
    losses = example().train(vocab=200, width=64, tokens=1024, steps=60)
    assert 4.5 < losses[0] < 7.0
    assert losses[-1] < 0.5 * losses[0]


def test_two_runs_same_bits():
    ex = example()
    a, b = (ex.train(vocab=130, width=48, tokens=257, steps=5) for _ in range(2))
    assert a == b
