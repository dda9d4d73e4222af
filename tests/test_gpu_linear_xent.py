"""Softmax cross entropy of a linear layer and its gradients on the GPU against
the definition in 64 bits.

Bounds.  BF16 products are exact in FP32 and the tensor core adds 16 of them per
step into an FP32 accumulator, losing at most 2^-22 of the terms' magnitude per
step (one truncation of the aligned products, one of the sum); FP32 operands
add the dropped plane products (4 * 2^-27) and five more passes of terms that are
2^-8 of the leading ones.  So a product over k is within
    (1.1 k / 16 + 8) 2^-22 + 2^-25
of sum |a||b|.  From there the errors follow the formulas.
"""
import ctypes

import pytest
import torch

from gpu_helpers import env
from train_helpers import TINY, U, close, directional, padded, untouched

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = U[F32]


@pytest.fixture(scope="module")
def b2g():
    return env()[1]


@pytest.fixture(autouse=True)
def clean_status(b2g):
    yield
    b2g.b2g_status(torch.cuda.current_stream().cuda_stream)


def status(b2g):
    return b2g.b2g_status(torch.cuda.current_stream().cuda_stream)


def prod(k):
    return (1.1 * k / 16 + 8) * 2.0 ** -22 + 2.0 ** -25


class Reference:
    def __init__(self, h, w, target, ignore):
        h, w = h.double(), w.double()
        z = h @ w.t()
        ez = prod(h.shape[1]) * (h.abs() @ w.abs().t())     # error of each logit
        self.valid = (target != ignore) & (target >= 0) & (target < w.shape[0])
        at = torch.where(self.valid, target.long(), torch.zeros_like(target.long()))[:, None]
        self.at, self.h, self.w = at, h, w
        self.lse = torch.logsumexp(z, 1)
        # the exponentials' 2^-22 and the rounding of their arguments, at most 256
        # sequential additions and the joins, and the logarithm's last bits
        self.elogit, self.elarg = ez, ez + 4 * U32 * (z - self.lse[:, None]).abs()
        self.elu = torch.logsumexp(z + self.elarg, 1) - self.lse + 2.0 ** -20 + 400 * U32 \
            + 4 * U32 * self.lse.abs() + TINY
        zt = z.gather(1, at)[:, 0]
        zero = torch.zeros_like(zt)
        nan = torch.full_like(zt, float("nan"))
        self.loss = torch.where(self.valid, self.lse - zt, torch.where(target == ignore, zero, nan))
        self.eloss = self.elu + ez.gather(1, at)[:, 0] + 2 * U32 * (self.lse.abs() + zt.abs())
        self.z = z

    def grads(self, g, lse, dtype):
        """dh, dw and their bounds, for the lse the backward call is given."""
        lse = lse.double()[:, None]
        g = torch.where(self.valid, g.double(), torch.zeros_like(g.double()))[:, None]
        p = torch.exp(self.z - lse)
        p = torch.where(self.valid[:, None], p, torch.zeros_like(p))
        dz = p * g
        # exp's argument carries the logit's error and its own rounding
        arg = self.z - lse
        ep = g.abs() * (torch.exp(arg + self.elogit + 4 * U32 * arg.abs()) - p + 2.0 ** -21 * p)
        dz.scatter_add_(1, self.at, -g)
        ep = torch.where(self.valid[:, None], ep + 2 * U32 * (dz.abs() + p * g.abs()),
                         torch.zeros_like(ep))
        ep += (U[BF16] if dtype is BF16 else 2.0 ** -25) * dz.abs()  # dz's rounding
        a = dz.abs() + ep
        dh, dw = dz @ self.w, dz.t() @ self.h
        bh = ep @ self.w.abs() + (prod(a.shape[1]) + 100 * U32) * (a @ self.w.abs())
        bw = ep.t() @ self.h.abs() + (prod(a.shape[0]) + 100 * U32) * (a.t() @ self.h.abs())
        return dh, bh, dw, bw


def make(tokens, vocab, width, dtype, seed=0, ignored=0.1):
    gen = torch.Generator().manual_seed(seed + tokens * 7 + vocab + width)
    w = torch.randn(vocab, width, generator=gen, dtype=torch.float64) * 0.3
    t = torch.randint(0, vocab, (tokens,), generator=gen)
    h = torch.randn(tokens, width, generator=gen, dtype=torch.float64)
    h[::2] += w[t[::2]]
    t[torch.rand(tokens, generator=gen) < ignored] = -100
    g = torch.rand(tokens, generator=gen) / tokens
    return h.to(dtype).cuda(), w.to(dtype).cuda(), t.cuda(), g.cuda()


def check(b2g, h, w, t, g, ignore=-100, **kw):
    loss, lse = b2g.linear_cross_entropy(h, w, t, ignore_index=ignore)
    ref = Reference(h, w, t, ignore)
    close(lse, ref.lse, ref.elu, "lse")
    close(loss, ref.loss, ref.eloss, "loss")
    old = kw["dw"].double() if kw.get("accumulate") else 0
    dh, dw = b2g.linear_cross_entropy_backward(h, w, t, lse, g, ignore_index=ignore, **kw)
    rh, bh, rw, bw = ref.grads(g, lse, h.dtype)
    u = U[h.dtype] * (1 + 1e-6)
    close(dh, rh, bh + u * rh.abs() + TINY, "dh")
    rw = rw + old
    close(dw, rw, bw + u * rw.abs() + 2 * U32 * rw.abs() + TINY, "dw")
    return loss, lse, dh, dw


SHAPES = [
    (1, 1, 1), (1, 2, 8), (3, 5, 7), (2, 257, 64), (129, 300, 65), (256, 256, 64), (257, 511, 130),
    (64, 1000, 33), (16, 5000, 512), (1, 40000, 256), (300, 700, 1000), (513, 1025, 264),
    (1000, 2048, 128), (130, 20001, 128), (5000, 130, 72), (64, 64, 8), (65, 300, 40), (33, 513, 136),
    (17, 20000, 72), (64, 3000, 520), (48, 40000, 64), (100, 100, 4104), (384, 4096, 777),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,width", SHAPES)
def test_forward_and_backward(b2g, tokens, vocab, width, dtype):
    h, w, t, g = make(tokens, vocab, width, dtype)
    check(b2g, h, w, t, g)
    assert status(b2g) == (0, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,width", [
    (65, 5207, 40), (66, 7310, 40), (67, 10114, 72), (65, 12217, 40), (70, 15021, 72), (65, 17124, 40),
    (300, 9000, 200), (500, 20001, 40)])
def test_widths_of_a_tile(b2g, tokens, vocab, width, dtype):
    """Tiles of 96, 128, 160, 192, 224 and 256 classes, the last one of a row ragged."""
    h, w, t, g = make(tokens, vocab, width, dtype)
    check(b2g, h, w, t, g)


@pytest.mark.parametrize("dtype,tokens,vocab,width", [
    (F32, 8192, 12000, 64), (BF16, 8192, 40000, 64), (F32, 64, 1500000, 8)])
def test_several_pieces_of_the_vocabulary(b2g, dtype, tokens, vocab, width):
    h, w, t, g = make(tokens, vocab, width, dtype)
    check(b2g, h, w, t, g)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_targets_as_int32_and_accumulation(b2g, dtype):
    h, w, t, g = make(200, 600, 96, dtype)
    dw = torch.randn(600, 96, dtype=torch.float64).to(dtype).cuda()
    check(b2g, h, w, t.int(), g, dw=dw, accumulate=True)
    h, w, t, g = make(3000, 70, 40, dtype)  # k slices of dw, added to its old values
    dw = torch.randn(70, 40, dtype=torch.float64).to(dtype).cuda()
    check(b2g, h, w, t, g, dw=dw, accumulate=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (8, 8), (3, 5)])
def test_strides_alignment_and_guards(b2g, extra, offset, dtype):
    h, w, t, g = make(150, 330, 104, dtype)
    hp, _ = padded(h.double().cpu(), dtype, 104 + extra, offset)
    wp, _ = padded(w.double().cpu(), dtype, 104 + extra, offset)
    dw, flat = padded(w.double().cpu(), dtype, 104 + extra, offset)
    before = flat.clone()
    check(b2g, hp, wp, t, g, dw=dw)
    assert untouched(flat, dw, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_without_a_target(b2g, dtype):
    h, w, t, g = make(140, 300, 64, dtype)
    t[:] = 7
    loss, lse, dh, dw = check(b2g, h, w, t, g, ignore=7)
    assert not loss.any() and not dh.any() and not dw.any()
    t[3] = 8
    loss, lse, dh, dw = check(b2g, h, w, t, g, ignore=7)
    assert dh[3].any() and not dh[4].any()


def test_targets_out_of_range(b2g):
    h, w, t, g = make(140, 300, 64, F32)
    t[5], t[6], t[139] = 300, -1, 1 << 40
    check(b2g, h, w, t, g)
    assert status(b2g) == (b2g.B2G_ERR_INDEX, 1 << 16)
    assert status(b2g) == (0, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_and_equal_logits(b2g, dtype):
    """Logits of thousands (exponentials far outside FP32), and a row of equal ones."""
    h, w, t, g = make(70, 500, 64, dtype, ignored=0)
    h[0] = 0
    h[1] *= 300
    h[2] *= -300
    loss, lse, dh, dw = check(b2g, h, w, t, g)
    assert abs(float(lse[0]) - 6.2146081) < 1e-5


def test_masked_classes(b2g):
    """A class whose logits are the type's lowest values has probability 0 and no
    gradient; every other class is as without it."""
    h, w, t, g = make(40, 100, 16, F32, ignored=0)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w[37:41] = 0
    w[37:41, 0] = -1e30
    t[(t >= 37) & (t < 41)] = 0
    loss, lse, dh, dw = check(b2g, h, w, t, g)
    assert torch.isfinite(loss).all() and not dw[37:41].any()


@pytest.mark.parametrize("tokens", [40, 130])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_classes_masked_by_the_lowest_value(b2g, tokens, dtype):
    """Logits of the type's lowest value, which FP32's BF16 planes must not round
    to infinity."""
    h, w, t, g = make(tokens, 700, 32, dtype, ignored=0)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w[600:605] = 0
    w[600:605, 0] = torch.finfo(dtype).min
    t[(t >= 600) & (t < 605)] = 0
    loss, lse, dh, dw = check(b2g, h, w, t, g)
    assert torch.isfinite(loss).all() and torch.isfinite(dh[:, 1:]).all()
    assert not dw[600:605].any()


def test_weights_of_zero_and_nonfinite_lse(b2g):
    """A row of weight 0 has no gradient, whatever its lse is."""
    h, w, t, g = make(33, 90, 24, F32, ignored=0)
    g[4] = 0
    _, lse = b2g.linear_cross_entropy(h, w, t)
    ref = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    lse[4] = float("nan")
    got = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    assert not ref[0][4].any() and all(torch.equal(p, q) for p, q in zip(ref, got))


@pytest.mark.parametrize("tokens", [40, 300])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_subnormal_weights(b2g, tokens, dtype):
    """Weights whose reciprocal is infinite, next to weights of exactly 0 and classes of
    probability 0: the gradients are finite, and 0 in the rows of weight 0."""
    h, w, t, g = make(tokens, 700, 32, dtype, ignored=0)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w[600:605] = 0
    w[600:605, 0] = torch.finfo(dtype).min
    t[(t >= 600) & (t < 605)] = 0
    g[:] = 2e-39
    g[::3] = 0
    _, _, dh, dw = check(b2g, h, w, t, g)
    assert torch.isfinite(dh[:, 1:]).all() and torch.isfinite(dw).all()
    assert not dh[::3].any() and dw[:, 1:].any()


@pytest.mark.parametrize("tokens", [40, 130])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weights_of_rows_without_a_gradient(b2g, tokens, dtype):
    """The weights of ignored and out-of-range rows are not looked at: any values there
    leave the other rows' gradients the bits they have with 0."""
    h, w, t, g = make(tokens, 700, 96, dtype, ignored=0)
    t[5], t[11], t[17] = -100, 700, -3
    g[[5, 11, 17]] = 0
    _, lse, dh, dw = check(b2g, h, w, t, g)
    for value in (1e38, float("inf"), float("nan"), 1e-30):
        g[[5, 11, 17]] = value
        got = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
        assert torch.equal(got[0], dh) and torch.equal(got[1], dw), value


def test_products_over_very_many_classes(b2g):
    """dh over 2^28 classes, whose terms all have one sign.  The tensor core truncates each
    addition (2^-23 of the sum at most), 2048 of them in a row before FP32 registers take
    over.  Every logit is 0 and each probability 2^-28 to 2^-18 (its exponential's error and
    that of lse), which rounds to BF16's 2^-28; the target's row of w is 0, so dh is the mean
    of w's rows."""
    vocab, width = 1 << 28, 8
    w = torch.empty(vocab, width, dtype=BF16, device="cuda")
    gen, mean = torch.Generator(device="cuda").manual_seed(0), 0
    for i in range(0, vocab, 1 << 25):
        w[i:i + (1 << 25)] = torch.rand(1 << 25, width, generator=gen, device="cuda") + 1
        if i == 0:
            w[77] = 0
        mean = mean + w[i:i + (1 << 25)].double().sum(0) / vocab
    h, t = torch.zeros(1, width, dtype=BF16, device="cuda"), torch.tensor([77], device="cuda")
    loss, lse = b2g.linear_cross_entropy(h, w, t)
    want = 28 * 0.6931471805599453
    assert abs(float(lse) - want) <= 2.0 ** -20 + 8 * U32 * want and float(loss) == float(lse)
    dh, dw = b2g.linear_cross_entropy_backward(h, w, t, lse, torch.ones(1, device="cuda"))
    close(dh[0], mean, (U[BF16] + 2048 * 2.0 ** -23 + 2.0 ** -18) * mean, "dh")
    assert not dw.any()  # h is 0


def test_no_tokens(b2g):
    h, w = torch.empty(0, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    t, e = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = b2g.linear_cross_entropy(h, w, t)
    assert loss.shape == lse.shape == (0,)
    dh, dw = b2g.linear_cross_entropy_backward(h, w, t, e, e)
    assert dh.shape == (0, 64) and not dw.any()
    dw = b2g.linear_cross_entropy_backward(h, w, t, e, e, dw=w.clone(), accumulate=True)[1]
    assert torch.equal(dw, w)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_every_run(b2g, dtype):
    h, w, t, g = make(700, 3000, 200, dtype)
    loss, lse = b2g.linear_cross_entropy(h, w, t)
    first = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    for _ in range(4):
        again = b2g.linear_cross_entropy(h, w, t)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        got = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
        assert all(torch.equal(p, q) for p, q in zip(first, got))


@pytest.mark.parametrize("dtype,tokens,vocab,width,accumulate", [
    (BF16, 100, 5000, 777, False), (BF16, 700, 20001, 1001, False), (F32, 1000, 11007, 777, False),
    (BF16, 100, 60000, 512, True), (F32, 200, 9000, 333, True)])
def test_gradients_that_leave_in_two_ways(b2g, dtype, tokens, vocab, width, accumulate):
    """One launch in which a warp's buffer takes tiles of dh for bulk-tensor stores and then
    tiles of dw that go out element by element (an odd width, or adding to BF16 values):
    the 64-bit bound, and the same bits every time."""
    h, w, t, g = make(tokens, vocab, width, dtype)
    old = w.flip(0).contiguous() * 1e-3
    given = {"dw": old.clone(), "accumulate": True} if accumulate else {}
    _, lse, dh, dw = check(b2g, h, w, t, g, **given)
    first = dh.clone(), dw.clone()
    for _ in range(40):
        given = {"dw": old.clone(), "accumulate": True} if accumulate else {}
        got = b2g.linear_cross_entropy_backward(h, w, t, lse, g, **given)
        assert all(torch.equal(p, q) for p, q in zip(first, got))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,width", [(40, 3000, 136), (300, 5000, 200), (700, 9000, 520)])
def test_one_gradient_alone(b2g, tokens, vocab, width, dtype):
    """dh or dw not wanted (NULL): the other one has the bits it has with both."""
    lib, code = b2g.train.train_library(), 0 if dtype is F32 else 1
    gen = torch.Generator().manual_seed(tokens)
    h = torch.randn(tokens, width, generator=gen).to(dtype).cuda()
    w = (torch.randn(vocab, width, generator=gen) * width ** -0.5).to(dtype).cuda()
    target = torch.randint(0, vocab, (tokens,), generator=gen).cuda()
    loss, lse = b2g.linear_cross_entropy(h, w, target)
    g = torch.full((tokens,), 1.0 / tokens, device="cuda")
    dh, dw = b2g.linear_cross_entropy_backward(h, w, target, lse, g)
    nb = ctypes.c_size_t()
    assert lib.b2g_linear_xent_workspace_size(code, tokens, vocab, width, h.data_ptr(), width,
                                              w.data_ptr(), width, 1, ctypes.byref(nb)) == 0
    ws = torch.empty(nb.value, dtype=torch.uint8, device="cuda")
    for want in ("dh", "dw"):
        out = torch.full_like(dh if want == "dh" else dw, float("nan"))
        p = out.data_ptr()
        rc = lib.b2g_linear_xent_backward(
            code, tokens, vocab, width, h.data_ptr(), width, w.data_ptr(), width,
            target.data_ptr(), 8, -100, lse.data_ptr(), g.data_ptr(), p if want == "dh" else None,
            width, 0, p if want == "dw" else None, width, ws.data_ptr(), nb.value,
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert torch.equal(out, dh if want == "dh" else dw), want
    assert status(b2g)[0] == 0


def test_gradient_against_differences(b2g):
    h, w, t, g = make(24, 60, 32, F32)
    _, lse = b2g.linear_cross_entropy(h, w, t)
    grads = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    eps = 2.0 ** -6
    ref = Reference(h, w, t, -100)
    for k, grad in enumerate(grads):
        u = torch.randn_like((h, w)[k])

        def loss(s):
            a = [h, w]
            a[k] = a[k] + s * u
            return float((b2g.linear_cross_entropy(a[0], a[1], t)[0].double() * g.double()).sum())

        diff, trunc = directional(loss, eps)
        noise = float((ref.eloss * g.double()).sum()) * 8 / eps
        want = float((grad.double() * u.double()).sum())
        assert abs(diff - want) <= trunc + noise, (k, diff, want, trunc, noise)


def test_other_stream_and_graph(b2g):
    h, w, t, g = make(300, 900, 128, BF16)
    ref = b2g.linear_cross_entropy(h, w, t)
    grads = b2g.linear_cross_entropy_backward(h, w, t, ref[1], g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, lse = b2g.linear_cross_entropy(h, w, t, stream=s)
    got = b2g.linear_cross_entropy_backward(h, w, t, lse, g, stream=s)
    s.synchronize()
    assert torch.equal(loss, ref[0]) and all(torch.equal(p, q) for p, q in zip(got, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = b2g.linear_cross_entropy(h, w, t)
        got = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, ref[0]) and all(torch.equal(p, q) for p, q in zip(got, grads))


def test_bounded_wait_reports(b2g):
    """With the copies stopped early the waits run out, the calls return and the
    status word says so; the next call works again."""
    h, w, t, g = make(64, 128, 1024, BF16)
    loss, lse = b2g.linear_cross_entropy(h, w, t)
    torch.cuda.synchronize()
    try:
        b2g.b2g_set_wait_limit_ns(2_000_000)
        b2g.b2g_debug_stop_after(3)
        b2g.linear_cross_entropy(h, w, t)
        rc, flags = status(b2g)
        assert rc == b2g.B2G_ERR_TIMEOUT and flags & 0xF
    finally:
        b2g.b2g_debug_stop_after(-1)
        b2g.b2g_set_wait_limit_ns(2_000_000_000)
    again = b2g.linear_cross_entropy(h, w, t)
    assert torch.equal(again[0], loss) and status(b2g) == (0, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab", [(40, 2000), (300, 1000)])
@pytest.mark.parametrize("stop", [1, 2, 7])
def test_bounded_waits_of_both_forms(b2g, tokens, vocab, dtype, stop):
    """The same for the loss and for the gradients, up to 64 tokens and in CTA pairs, the
    copies stopped within and after a k tile's planes."""
    h, w, t, g = make(tokens, vocab, 1024, dtype)
    loss, lse = b2g.linear_cross_entropy(h, w, t)
    first = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    torch.cuda.synchronize()
    for call in (lambda: b2g.linear_cross_entropy(h, w, t),
                 lambda: b2g.linear_cross_entropy_backward(h, w, t, lse, g)):
        try:
            b2g.b2g_set_wait_limit_ns(2_000_000)
            b2g.b2g_debug_stop_after(stop)
            call()
            rc, flags = status(b2g)
            assert rc == b2g.B2G_ERR_TIMEOUT and flags & 0xF
        finally:
            b2g.b2g_debug_stop_after(-1)
            b2g.b2g_set_wait_limit_ns(2_000_000_000)
    again = b2g.linear_cross_entropy(h, w, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    got = b2g.linear_cross_entropy_backward(h, w, t, lse, g)
    assert all(torch.equal(p, q) for p, q in zip(first, got)) and status(b2g) == (0, 0)
