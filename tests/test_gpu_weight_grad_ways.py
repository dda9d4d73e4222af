"""Every way in which the weight gradient shares out its tiles: whole ones in rounds of the 76 CTA
pairs; the rest whole or halved, cut into slices, or into pieces that lie across two tiles;
few or many sums a tile for the launch that joins them; x prepared or read from its codes."""
import ctypes

import pytest
import torch

from test_gpu_weight_grad import check

F32, BF16 = torch.float32, torch.bfloat16
P = 0x100000  # an aligned address
PAIRS = 76


def up(v, n):
    return -(-v // n) * n


def way(lib, dtype, tokens, outs, width):
    """(x "codes" or "prepared", rounds of whole tiles, "slices", "across" or "whole", sums of a
    tile), from the bytes of workspace that the library asks for; of sizes whose copies' bytes are
    not a multiple of the sums'."""
    n = ctypes.c_size_t()
    assert lib.b2g_linear_dweight8_workspace_size_ex(0 if dtype is F32 else 1, tokens, outs, width, P, up(outs, 8),
                                                     P, up(width, 16), ctypes.byref(n)) == 0
    tile_n = 256 if width > 128 else 128
    rounds, rest = divmod(-(-outs // 256) * -(-width // tile_n), PAIRS)
    k_tiles = -(-tokens // 64)
    sums = 2 * 256 * tile_n * 4  # of a piece: two, where it lies across two tiles
    copies = up(tokens * up(width, 64) * 2, 256)
    if dtype is F32:
        copies += up(3 * tokens * up(outs, 64) * 2, 256)
    assert copies % sums != 0
    codes = dtype is BF16 and n.value % sums == 0
    pieces, odd = divmod(n.value - (0 if codes else copies), sums)
    assert odd == 0 and pieces >= 0
    if pieces == 0:
        kind, each = "whole", 0
    elif pieces % rest == 0:
        kind, each = "slices", pieces // rest
    else:  # one piece a pair, of as many k tiles as make `pieces` of all; one more where it is cut
        kind = "across"
        length = -(-rest * k_tiles // PAIRS)
        assert pieces == -(-rest * k_tiles // length)
        each = max((t * k_tiles + k_tiles - 1) // length - t * k_tiles // length + 1 for t in range(rest))
    return "codes" if codes else "prepared", rounds, kind, each


CASES = [
    (BF16, 15261, 312, 2544, ("codes", 0, "across", 5)), (BF16, 5983, 208, 4965, ("codes", 0, "across", 5)),
    (BF16, 734, 287, 232, ("codes", 0, "slices", 12)), (BF16, 537, 256, 256, ("codes", 0, "slices", 9)),
    (BF16, 61, 2872, 4744, ("codes", 3, "whole", 0)), (BF16, 300, 2872, 4744, ("prepared", 3, "whole", 0)),
    (BF16, 11580, 264, 3608, ("prepared", 0, "across", 4)), (BF16, 7453, 312, 3166, ("prepared", 0, "across", 4)),
    (BF16, 4345, 773, 262, ("prepared", 0, "slices", 7)), (BF16, 8372, 624, 320, ("prepared", 0, "slices", 11)),
    (BF16, 6065, 2176, 3238, ("prepared", 1, "across", 3)), (BF16, 7915, 1056, 6232, ("prepared", 1, "across", 3)),
    (BF16, 1407, 1368, 3297, ("prepared", 1, "slices", 8)), (BF16, 1567, 2608, 1552, ("prepared", 1, "slices", 13)),
    (BF16, 5924, 3712, 3138, ("prepared", 2, "across", 3)), (BF16, 1262, 5816, 2552, ("prepared", 3, "slices", 7)),
    (F32, 1833, 231, 6568, ("prepared", 0, "across", 4)), (F32, 1533, 5009, 291, ("prepared", 0, "across", 3)),
    (F32, 18697, 220, 1753, ("prepared", 0, "across", 12)),
    (F32, 440, 220, 368, ("prepared", 0, "slices", 7)), (F32, 133, 4096, 4090, ("prepared", 3, "whole", 0)),
    (F32, 663, 207, 205, ("prepared", 0, "slices", 11)), (F32, 2171, 7427, 1000, ("prepared", 1, "across", 3)),
    (F32, 1703, 4945, 1369, ("prepared", 1, "across", 3)), (F32, 334, 2513, 1968, ("prepared", 1, "slices", 6)),
    (F32, 615, 554, 6449, ("prepared", 1, "slices", 10)), (F32, 1538, 3867, 2969, ("prepared", 2, "across", 3)),
    (F32, 609, 5201, 2562, ("prepared", 3, "slices", 10)),
]


@pytest.fixture(scope="module")
def b2g():
    from dense_fp32_gemm_07_gb300 import build

    build.build()
    import dense_fp32_gemm_07_gb300 as pkg

    pkg.train_library()
    return pkg


@pytest.mark.parametrize("dtype,tokens,outs,width,expected", CASES)
def test_the_way_is_taken(b2g, dtype, tokens, outs, width, expected):
    """The sizes below keep covering the ways that they were chosen for."""
    assert way(b2g.train_library(), dtype, tokens, outs, width) == expected


def test_ways_are_all_there():
    seen = {(c[0], c[4][0], c[4][1] > 0, c[4][2], c[4][3] > 8) for c in CASES}
    for dtype in (F32, BF16):
        for rounds in (False, True):
            for kind, many in (("slices", False), ("slices", True), ("across", False)):
                assert (dtype, "prepared", rounds, kind, many) in seen
    assert {("across", False), ("slices", True)} <= {w[3:] for w in seen if w[1] == "codes"}
    assert (F32, "prepared", False, "across", True) in seen


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tokens,outs,width,expected", CASES)
def test_against_64_bits(b2g, dtype, tokens, outs, width, expected):
    """Into a new result, added to one, and into rows off the 16-byte boundaries between guards."""
    torch.manual_seed(tokens + outs + width)
    ldy = up(outs, 8)
    dy = torch.randn(tokens, ldy, device="cuda").to(dtype)[:, :outs]
    kept = b2g.quantize_8bit(torch.randn(tokens, width, device="cuda"))
    x = b2g.dequantize_8bit(*kept, F32)
    dw = b2g.linear_weight_grad_8bit(dy, *kept)
    check(dw, dy, x)
    old = torch.randn(outs, width, device="cuda").to(dtype)
    got = old.clone()
    assert b2g.linear_weight_grad_8bit(dy, *kept, dw=got, accumulate=True) is got
    check(got, dy, x, old)
    flat = torch.full((outs + 2, width + 3), 7.0, dtype=dtype, device="cuda")
    inside = flat[1:-1, 1:-2]
    b2g.linear_weight_grad_8bit(dy, *kept, dw=inside)
    assert torch.equal(inside, dw)
    inside.fill_(7.0)  # what is left are the guards
    assert (flat == 7.0).all()
