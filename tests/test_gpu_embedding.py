"""Embedding lookup and its gradient on the GPU against 64-bit sums."""
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


def check_forward(b2g, ids, table, scale, **kw):
    out = b2g.embedding(ids, table, scale=scale, **kw)
    want = table.double()[ids.long()] * float(torch.tensor(scale, dtype=F32))
    # one product in FP32, one rounding to the type
    close(out, want, (U[table.dtype] + U32) * want.abs() * 1.001 + TINY, "out")
    return out


def check_backward(b2g, ids, dout, vocab, scale=1.0, before=None, pad=None, **kw):
    got = b2g.embedding_backward(ids, dout, vocab, scale=scale, padding_idx=pad, **kw)
    ids = ids.long()
    keep = (ids >= 0) & (ids < vocab)
    if pad is not None:
        keep &= ids != pad
    d, at = dout.double()[keep], ids[keep]
    s = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device="cuda").index_add_(0, at, d)
    a = torch.zeros_like(s).index_add_(0, at, d.abs())
    n = torch.zeros(vocab, device="cuda", dtype=torch.float64).index_add_(
        0, at, torch.ones(len(at), device="cuda", dtype=torch.float64))[:, None]
    sc = float(torch.tensor(scale, dtype=F32))
    want = s * sc + (0 if before is None else before.double())
    # a run of n rows: at most n - 1 rounded additions on the way of any row, the
    # scaling and the addition of the old value
    bound = (n + 2) * U32 * a * abs(sc) + 2 * U32 * want.abs() \
        + U[dout.dtype] * want.abs() * (1 + 1e-6) + TINY
    if before is not None:
        bound = torch.where(n > 0, bound, torch.zeros_like(bound))  # untouched rows keep their bits
    close(got, want, bound, "dtable")
    return got


CASES = [
    # tokens, vocab, width
    (1, 1, 1), (1, 7, 64), (2, 3, 5), (15, 4, 8), (16, 1000, 128), (17, 40, 33), (31, 300, 256),
    (257, 50, 129), (1000, 70000, 24), (2048, 17, 512), (4095, 5003, 100), (4097, 33, 40),
    (20000, 300, 16), (40001, 70001, 8), (128, 129, 4096), (33, 12, 9000),
    (33000, 300001, 4),  # three digits
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,vocab,width", CASES)
def test_forward_and_backward(b2g, tokens, vocab, width, dtype):
    gen = torch.Generator().manual_seed(tokens + vocab + width)
    ids = torch.randint(0, vocab, (tokens,), generator=gen).cuda()
    table = torch.randn(vocab, width, generator=gen).to(dtype).cuda()
    dout = torch.randn(tokens, width, generator=gen).to(dtype).cuda()
    check_forward(b2g, ids, table, 1.75)
    check_backward(b2g, ids, dout, vocab, 1.75)
    check_backward(b2g, ids.int(), dout, vocab)
    before = torch.randn(vocab, width, generator=gen).to(dtype).cuda()
    check_backward(b2g, ids, dout, vocab, -0.5, before=before, out=before.clone(), accumulate=True)
    assert status(b2g) == (0, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [5, 16, 17, 300, 5000, 33000])
def test_one_token_repeated(b2g, tokens, dtype):
    """One run through every window, with and without a neighbour on each side."""
    dout = torch.randn(tokens, 72, device="cuda").to(dtype)
    ids = torch.full((tokens,), 3, device="cuda")
    check_backward(b2g, ids, dout, 9)
    ids[0], ids[-1] = 0, 8
    check_backward(b2g, ids, dout, 9)
    ids[tokens // 2] = 2
    check_backward(b2g, ids, dout, 9)


def test_runs_at_window_edges(b2g):
    """Run lengths around the window size, so that runs end at, before and after edges."""
    lens = [1, 15, 16, 17, 31, 32, 33, 16, 16, 1, 1, 48, 127, 128, 129, 2, 14, 16, 240, 1]
    ids = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)])
    dout = torch.randn(len(ids), 36, dtype=torch.float64)
    perm = torch.randperm(len(ids))
    for order in (torch.arange(len(ids)), perm):
        check_backward(b2g, ids[order].cuda(), dout[order].float().cuda(), len(lens) + 3)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_frequent_and_rare_tokens(b2g, dtype):
    gen = torch.Generator().manual_seed(5)
    u = torch.rand(30000, generator=gen, dtype=torch.float64)
    ids = (torch.exp(u * 11.0).long() - 1).cuda()
    dout = torch.randn(30000, 64, generator=gen).to(dtype).cuda()
    a = check_backward(b2g, ids, dout, 60000)
    for _ in range(3):
        assert torch.equal(a, b2g.embedding_backward(ids, dout, 60000))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (5, 3), (8, 8)])
def test_strides_alignment_and_guards(b2g, extra, offset, dtype):
    gen = torch.Generator().manual_seed(extra * 10 + offset)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    ids = torch.randint(0, 50, (90,), generator=gen).cuda()
    table, _ = padded(mk(50, 96), dtype, 96 + extra, offset)
    out, flat = padded(mk(90, 96), dtype, 96 + extra, offset)
    before = flat.clone()
    check_forward(b2g, ids, table, 0.5, out=out)
    assert untouched(flat, out, before)
    dt, flat = padded(mk(50, 96), dtype, 96 + extra, offset)
    before = flat.clone()
    check_backward(b2g, ids, out, 50, out=dt)
    assert untouched(flat, dt, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,width,ldt,ldo,ot,oo", [
    (5000, 257, 257, 257, 0, 0), (5000, 257, 260, 263, 1, 3), (700, 2001, 2001, 2003, 2, 1),
    (30000, 43, 43, 43, 1, 0), (20000, 70, 71, 72, 0, 2)])
def test_large_lookup_at_any_alignment(b2g, tokens, width, ldt, ldo, ot, oo, dtype):
    """Lookups off the 16-byte boundaries, in words of the output row; ids out of range."""
    gen = torch.Generator().manual_seed(width + ot)
    vocab = 500
    ids = torch.randint(0, vocab, (tokens,), generator=gen).cuda()
    table, _ = padded(torch.randn(vocab, width, generator=gen, dtype=torch.float64), dtype, ldt, ot)
    out, flat = padded(torch.zeros(tokens, width, dtype=torch.float64), dtype, ldo, oo)
    before = flat.clone()
    check_forward(b2g, ids, table, -0.75, out=out)
    assert untouched(flat, out, before)
    assert status(b2g)[0] == 0
    bad = ids.clone()
    bad[3], bad[tokens - 1] = -1, vocab
    got = b2g.embedding(bad, table, out=out)
    assert torch.isnan(got[3]).all() and torch.isnan(got[-1]).all()
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[3] = keep[-1] = False
    assert torch.equal(got[keep], table[ids[keep]])
    assert status(b2g)[0] == b2g.B2G_ERR_INDEX


def test_padding_and_out_of_range(b2g):
    table, dout = torch.randn(10, 32, device="cuda"), torch.randn(6, 32, device="cuda")
    ids = torch.tensor([4, 0, 9, 4, 0, 2], device="cuda")
    check_backward(b2g, ids, dout, 10, pad=4)
    assert status(b2g) == (0, 0)
    bad = torch.tensor([4, -1, 9, 10, 1 << 40, 2], device="cuda")
    out = b2g.embedding(bad, table)
    assert status(b2g) == (b2g.B2G_ERR_INDEX, 1 << 16)
    ok = torch.tensor([0, 2, 5])
    assert torch.equal(out[ok], table[bad[ok]])
    assert torch.isnan(out[torch.tensor([1, 3, 4])]).all()
    check_backward(b2g, bad, dout, 10)
    assert status(b2g) == (b2g.B2G_ERR_INDEX, 1 << 16)
    assert status(b2g) == (0, 0)


def test_no_tokens(b2g):
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    table = torch.randn(5, 16, device="cuda")
    assert b2g.embedding(ids, table).shape == (0, 16)
    e = torch.empty(0, 16, device="cuda")
    assert not b2g.embedding_backward(ids, e, 5).any()
    assert torch.equal(b2g.embedding_backward(ids, e, 5, out=table.clone(), accumulate=True), table)


def test_nonfinite_rows_stay_in_their_row(b2g):
    dout = torch.ones(40, 24, device="cuda")
    dout[7] = float("inf")
    dout[8, 3] = float("nan")
    ids = torch.arange(40, device="cuda") % 20
    g = b2g.embedding_backward(ids, dout, 21)
    assert torch.isinf(g[7]).all() and torch.isnan(g[8, 3])
    rest = torch.ones_like(g, dtype=torch.bool)
    rest[7], rest[8, 3] = False, False
    assert torch.isfinite(g[rest]).all()


def test_gradient_against_differences(b2g):
    """The lookup is linear in the table, so central differences are exact up to
    rounding."""
    torch.manual_seed(1)
    table, u = torch.randn(30, 20, device="cuda"), torch.randn(30, 20, device="cuda")
    ids = torch.randint(0, 30, (200,), device="cuda")
    dout = torch.randn(200, 20, device="cuda")
    g = b2g.embedding_backward(ids, dout, 30, scale=3.0)

    def loss(t):
        return float((b2g.embedding(ids, table + t * u, scale=3.0).double() * dout.double()).sum())

    diff, trunc = directional(loss, 0.5)
    size = float((dout.double().abs() * 3 * (table.abs() + u.abs()).double()[ids]).sum())
    want = float((g.double() * u.double()).sum())
    assert abs(diff - want) <= trunc + 200 * U32 * size


def test_offsets_past_32_bits(b2g):
    """A table of 2^32 + elements: the last rows' offsets need 64 bits."""
    vocab, width = 140000, 32768
    table = torch.empty(vocab, width, dtype=BF16, device="cuda")
    ids = torch.tensor([0, vocab - 1, 131072, vocab - 2], device="cuda")
    for i in ids.tolist():
        table[i] = torch.randn(width, device="cuda").to(BF16)
    out = check_forward(b2g, ids, table[:, :], 1.0)
    before = table[ids].clone()
    b2g.embedding_backward(ids, out, vocab, out=table, accumulate=True)
    want = before.double() * 2
    close(table[ids], want, U[BF16] * want.abs(), "dtable")


@pytest.mark.parametrize("width", [65536 * 256 + 8, 65535 * 256 + 1])
def test_gradient_of_very_wide_rows(b2g, width):
    """More than 65535 blocks of columns, on and off the 16-byte boundaries, and a run that
    two windows share.  Whole numbers: every FP32 sum is exact."""
    tokens = 130
    dout = torch.randint(-4, 5, (tokens, width), device="cuda", dtype=torch.int8).bfloat16()
    ids = torch.full((tokens,), 2, device="cuda")
    ids[:3] = 0
    got = b2g.embedding_backward(ids, dout, 4)
    assert status(b2g) == (0, 0)
    for c in range(0, width, 1 << 21):
        part = dout[:, c:c + (1 << 21)]
        assert torch.equal(got[0, c:c + (1 << 21)], part[:3].float().sum(0).bfloat16())
        assert torch.equal(got[2, c:c + (1 << 21)], part[3:].float().sum(0).bfloat16())
    assert not got[1].any() and not got[3].any()


def test_lookup_of_very_wide_rows(b2g):
    width = 65535 * 4096 + 4
    table = torch.empty(2, width, device="cuda")
    table[0], table[1] = 1.0, 2.0
    table[:, -5:] = torch.arange(10, device="cuda").view(2, 5).float()
    out = b2g.embedding(torch.tensor([1, 0], device="cuda"), table, scale=0.5)
    assert status(b2g) == (0, 0)
    assert torch.equal(out, table.flip(0) * 0.5)
