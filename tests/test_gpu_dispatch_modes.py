"""The tensor calls under torch's dispatch modes, profiler and deterministic filling: their
results are allocated where those see it, and are the same bits as otherwise."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gpu_helpers import env

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


class Seen(TorchDispatchMode):
    """Counts the tensors that come from torch's allocating operators."""

    def __init__(self):
        super().__init__()
        self.empty = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.empty += "empty" in str(func)
        return func(*args, **(kwargs or {}))


def calls(b2g):
    """(name, call, the least number of allocations) of each operator with plain arguments."""
    torch.manual_seed(1)
    x, dy = (torch.randn(40, 48, device="cuda") for _ in range(2))
    w = torch.randn(48, device="cuda")
    ids = torch.randint(0, 40, (30,), device="cuda")
    target = torch.randint(0, 40, (40,), device="cuda")
    _, mean, rstd = b2g.layer_norm(x, w, w)
    _, lse = b2g.linear_cross_entropy(dy, x, target)
    each = torch.rand(40, device="cuda")
    _, _, rms = b2g.rms_norm(x, w)
    kept = b2g.quantize_8bit(x)
    return [
        ("layer_norm", lambda: b2g.layer_norm(x, w, w), 3),
        ("layer_norm_backward", lambda: b2g.layer_norm_backward(dy, x, w, mean, rstd), 3),
        ("embedding", lambda: b2g.embedding(ids, x), 1),
        ("embedding_backward", lambda: b2g.embedding_backward(ids, x[:30], 40), 1),
        ("linear_cross_entropy", lambda: b2g.linear_cross_entropy(dy, x, target), 2),
        ("linear_cross_entropy_backward",
         lambda: b2g.linear_cross_entropy_backward(dy, x, target, lse, each), 2),
        ("grad_norm", lambda: b2g.grad_norm([x, w]), 1),
        ("rms_norm", lambda: b2g.rms_norm(x, w, dy), 3),
        ("rms_norm_8bit", lambda: b2g.rms_norm_8bit(x, w, dy, with_y=True, keep_total=True), 7),
        ("rms_norm_backward", lambda: b2g.rms_norm_backward(dy, x, w, rms, dy), 2),
        ("rms_norm_backward from 8 bits", lambda: b2g.rms_norm_backward(dy, kept, w, rms), 2),
        ("quantize_8bit", lambda: b2g.quantize_8bit(x), 2),
        ("dequantize_8bit", lambda: b2g.dequantize_8bit(*kept), 1),
        ("linear_weight_grad_8bit", lambda: b2g.linear_weight_grad_8bit(dy, *kept), 1),
    ]


def flat(v):
    if isinstance(v, torch.Tensor):
        return [v.reshape(-1).view(torch.uint8)]
    return [t for e in v or () for t in flat(e)]


def same(a, b):
    a, b = flat(a), flat(b)
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_modes_see_the_results(b2g):
    for name, call, least in calls(b2g):
        want = call()
        with Seen() as seen:
            got = call()
        assert seen.empty >= least, (name, seen.empty)
        assert same(got, want), name


def test_profiler_sees_the_results(b2g):
    for name, call, least in calls(b2g):
        call()
        with torch.autograd.profiler.profile() as p:
            call()
        n = sum(e.count for e in p.key_averages() if e.key.startswith("aten::empty"))
        assert n >= least, (name, n)


def test_deterministic_filling(b2g):
    """Memory that a call leaves as it was (behind the codes of a row) holds torch's filling."""
    x = torch.randn(40, 35, device="cuda")
    want = b2g.quantize_8bit(x)
    try:
        torch.use_deterministic_algorithms(True)
        filling = torch.empty(1, dtype=torch.float8_e4m3fn, device="cuda").view(torch.uint8)
        codes, scales = b2g.quantize_8bit(x)
        behind = codes.as_strided((40, 48), (48, 1)).view(torch.uint8)[:, 35:]
        assert (behind == filling).all() and same((codes, scales), want)
        for name, call, _ in calls(b2g):
            call()
    finally:
        torch.use_deterministic_algorithms(False)
