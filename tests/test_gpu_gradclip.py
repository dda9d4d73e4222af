"""The global gradient norm and clipping on the GPU against 64-bit results."""
import math

import pytest
import torch

from gpu_helpers import env
from train_helpers import TINY, U, close, directional

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = U[F32]


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


def gamma(n):
    """A thread adds at most 64 squares per chunk over its chunks, then 5 + 5
    levels of pairs, then the blocks' sums: at most 2 per thread and 10 levels per
    608 of them, every sum of positive terms.  The root halves the relative error."""
    per_thread = 64 * (1 + n / (608 * 2048))
    return (per_thread + 10 + 16 + 2) * U32 / 2 + 2 * U32


def check(b2g, grads, max_norm, outs=None):
    n = sum(g.numel() for g in grads)
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    originals = [g.clone() for g in grads]
    assert abs(float(b2g.grad_norm(grads)) - want) <= gamma(n) * want + TINY
    norm = b2g.clip_grad_norm(grads, max_norm, out=outs)
    assert norm.shape == () and norm.dtype is F32
    assert abs(float(norm) - want) <= gamma(n) * want + TINY
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(originals, grads if outs is None else outs):
        w = g.double() * coef
        close(o, w, (gamma(n) + 4 * U32 + U[g.dtype]) * w.abs() * 1.001 + TINY, "clipped")
    if outs is not None:
        assert all(torch.equal(g, o) for g, o in zip(grads, originals))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [
    [1], [7], [0, 5, 0], [2048], [2049, 1], [4096, 4097, 3], [16384 * 3 + 5], [100] * 7,
    [1025, 129, 33, 17, 1, 2, 3] * 20, [3] * 250, [1 << 20, 5, (1 << 19) + 3],
])
@pytest.mark.parametrize("where", ["in place", "apart"])
def test_norm_and_clip(b2g, sizes, dtype, where):
    gen = torch.Generator().manual_seed(sum(sizes))
    grads = [torch.randn(n, generator=gen).to(dtype).cuda() for n in sizes]
    outs = [torch.full_like(g, 9.0) for g in grads] if where == "apart" else None
    check(b2g, grads, 0.25 * math.sqrt(sum(sizes)), outs)
    check(b2g, grads, 1e9, outs)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_views_of_one_buffer(b2g, dtype, shift):
    """Views at every alignment; the results' alignment is the same or another one."""
    sizes = [33, 1, 16, 4099, 7, 20000]
    flat = torch.randn(sum(sizes) + 8, device="cuda").to(dtype)
    outf = torch.full((sum(sizes) + 8,), 5.0, device="cuda").to(dtype)
    grads = list(flat[1:1 + sum(sizes)].split(sizes))
    outs = list(outf[1 + shift:1 + shift + sum(sizes)].split(sizes))
    check(b2g, grads, 3.0, outs)
    assert (outf[:1 + shift] == 5).all() and (outf[1 + shift + sum(sizes):] == 5).all()


def test_shapes_of_tensors(b2g):
    check(b2g, [torch.randn(3, 5, 7, device="cuda"), torch.randn((), device="cuda"),
                torch.randn(2, 1, device="cuda")], 0.5)


@pytest.mark.parametrize("value,factor", [(float("inf"), 0.0), (float("nan"), float("nan"))])
def test_nonfinite(b2g, value, factor):
    a, b = torch.ones(3000, device="cuda"), torch.ones(5, device="cuda")
    b[2] = value
    norm = b2g.clip_grad_norm([a, b], 1.0)
    assert torch.equal(torch.isnan(norm).cpu(), torch.tensor(math.isnan(value)))
    assert math.isnan(value) or math.isinf(float(norm))
    if math.isnan(factor):
        assert torch.isnan(a).all() and torch.isnan(b).all()
    else:
        assert not a.any() and torch.isnan(b[2]) and not b[[0, 1, 3, 4]].any()


def test_zero_gradients_and_zero_limit(b2g):
    a = [torch.zeros(100, device="cuda")]
    assert float(b2g.clip_grad_norm(a, 1.0)) == 0 and not a[0].any()
    a = [torch.ones(100, device="cuda")]
    assert float(b2g.clip_grad_norm(a, 0.0)) == 10 and not a[0].any()


def test_same_bits_every_run(b2g):
    grads = [torch.randn(n, device="cuda") for n in (100001, 77, 2000003)]
    first = b2g.grad_norm(grads)
    assert all(torch.equal(first, b2g.grad_norm(grads)) for _ in range(5))


def test_norm_against_differences(b2g):
    """d norm / d t along u is <x, u> / norm."""
    torch.manual_seed(0)
    x, u = torch.randn(5000, device="cuda"), torch.randn(5000, device="cuda")
    n = float(b2g.grad_norm([x]))
    diff, trunc = directional(lambda t: float(b2g.grad_norm([x + t * u])), 0.25)
    want = float((x.double() * u.double()).sum()) / n
    assert abs(diff - want) <= trunc + 4 * (gamma(5000) + 2 * U32) * n / 0.25


def test_captured_in_a_graph(b2g):
    """Addresses travel in the launch, so a graph replays them on new values."""
    grads = [torch.randn(5000, device="cuda"), torch.randn(31, device="cuda")]
    outs = [torch.empty_like(g) for g in grads]
    b2g.clip_grad_norm(grads, 1.0, out=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = b2g.clip_grad_norm(grads, 1.0, out=outs)
    for t in grads:
        t.copy_(torch.randn_like(t))
    g.replay()
    ref = b2g.clip_grad_norm(grads, 1.0, out=[torch.empty_like(t) for t in grads])
    assert torch.equal(norm, ref)


def test_overlapping_results_are_refused(b2g):
    """A result that shares memory with another one, or with a tensor other than its own,
    on the current stream and on another one; what does not overlap is served."""
    flat = torch.arange(1.0, 101.0, device="cuda")
    a, b, c = flat[:40], flat[40:60], flat[60:]
    other = torch.zeros(100, device="cuda")
    empty = torch.empty(0, device="cuda")
    before = flat.clone()
    bad = [
        ([a, b, a], None),                            # the same tensor twice, in place
        ([flat, b], None),                            # a tensor and a part of it
        ([a, b], [other[:40], other[30:50]]),         # two results
        ([a, b], [flat[1:41], other[:20]]),           # a result one element past its tensor
        ([b, flat[80:]], [flat[80:], other[:20]]),    # another tensor's memory
        ([a, a], [a, other[:40]]),                    # in place, and still read as the other
        ([b, a, empty], [other[:20], flat[20:60], empty]),
    ]
    for stream in (None, torch.cuda.Stream()):
        for grads, out in bad:
            with pytest.raises(ValueError, match="overlap"):
                b2g.clip_grad_norm(grads, 1.0, out=out, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and not other.any()
    for grads, out in (([c, a, empty, b], None), ([a, b], [a, other[:20]]),
                       ([a, a], [other[:40], other[50:90]]), ([b, a], [other[:20], a])):
        check(b2g, [g.clone() for g in grads] if out is None else grads, 1e9, out)
        b2g.clip_grad_norm(grads, 1e9, out=out)
    assert torch.equal(flat, before)
    assert float(b2g.grad_norm([a, a])) > 0           # the norm only reads


def test_lists_of_other_things_are_refused(b2g):
    """A parameter without a gradient leaves a None in the list."""
    x = torch.ones(5, device="cuda")
    for call in (lambda: b2g.grad_norm([x, None]), lambda: b2g.clip_grad_norm([None, x], 1.0),
                 lambda: b2g.clip_grad_norm([x, x.bfloat16()], 1.0),
                 lambda: b2g.clip_grad_norm([x], 1.0, out=[None]),
                 lambda: b2g.clip_grad_norm([x], 1.0, out=[x.tolist()])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        b2g.clip_grad_norm([x, x.cpu()], 1.0)
