"""The 8-bit form of rows, from its definition in 64 bits: every code's value in a table,
the nearest one by comparison, scales by whole exponents."""
import math

import torch

BLOCK, LARGEST, LEAST = 32, 448.0, -110


def _magnitudes():
    """Values of the codes 0 .. 126: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


MAG = _magnitudes()


def values(codes, scales):
    """codes * scales in 64 bits, from the bytes."""
    c = codes.cpu().contiguous().view(torch.uint8).long()
    s = scales.cpu().contiguous().view(torch.uint8).double()
    table = torch.cat([MAG, torch.tensor([math.nan], dtype=torch.float64)])
    v = table[c & 127] * torch.where(c >= 128, -1.0, 1.0).double()
    s = torch.where(s == 255, torch.full_like(s, math.nan), torch.exp2(s - 127))
    return v * s.repeat_interleave(BLOCK, 1)[:, :c.shape[1]]


def exponent(largest):
    """The scale's exponent for a block's largest finite magnitude."""
    if largest == 0:
        return LEAST
    m, e = math.frexp(largest)                 # largest = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return max(LEAST, e - 9 + (1 if m > 0.875 else 0))


def encode(x):
    """(codes, scale bytes) as uint8 tensors of a matrix of any floating type."""
    x = x.double().cpu()
    r, c = x.shape
    nb = -(-c // BLOCK)
    b = torch.zeros(r, nb * BLOCK, dtype=torch.float64)
    b[:, :c] = x
    b = b.view(r, nb, BLOCK)
    size = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(2)
    e = torch.tensor([[exponent(float(v)) for v in row] for row in size],
                     dtype=torch.float64).view(r, nb)
    v = (b / torch.exp2(e)[:, :, None]).view(r, nb * BLOCK)[:, :c]
    a = torch.where(torch.isfinite(v), v.abs(), 0.0)
    hi = torch.searchsorted(MAG, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = MAG[hi] - a, a - MAG[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.isfinite(v), code, 127)
    sign = torch.where(torch.signbit(x) & torch.isfinite(v), 128, 0)
    return (code + sign).to(torch.uint8), (e + 127).to(torch.uint8)


def make(x, offset=0, ld=None, lds=None):
    """x's form as CUDA tensors of the types that the package uses, rows `ld` and `lds`
    bytes apart (None: on 16-byte boundaries; contiguous), the codes `offset` bytes past one."""
    codes, scales = encode(x)
    r, c = codes.shape
    nb = scales.shape[1]
    ld, lds = ld or -(-c // 16) * 16, lds or nb
    q = torch.full((offset + r * ld + 16,), 0x7f, dtype=torch.uint8, device="cuda")
    s = torch.full((r * lds + 16,), 255, dtype=torch.uint8, device="cuda")
    qv, sv = torch.as_strided(q, (r, c), (ld, 1), offset), torch.as_strided(s, (r, nb), (lds, 1), 0)
    qv.copy_(codes)
    sv.copy_(scales)
    return (torch.as_strided(q.view(torch.float8_e4m3fn), (r, c), (ld, 1), offset),
            torch.as_strided(s.view(torch.float8_e8m0fnu), (r, nb), (lds, 1), 0))


def same_bytes(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))
