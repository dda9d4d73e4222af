"""The weight gradient's workspace: no copy of x where it is read from its codes, and no
more than the query names."""
import ctypes

import pytest
import torch

P = 0x100000  # an aligned address


@pytest.fixture(scope="module")
def lib():
    from dense_fp32_gemm_07_gb300 import build

    build.build()
    import dense_fp32_gemm_07_gb300 as pkg

    return pkg.train_library()


def asked(lib, dtype, tokens, outs, width, dy=P, lddy=None, codes=P, ldq=None):
    """(bytes for any codes, bytes for these)."""
    any_, these = ctypes.c_size_t(), ctypes.c_size_t()
    lddy, ldq = lddy or -(-outs // 8) * 8, ldq or -(-width // 16) * 16
    assert lib.b2g_linear_dweight8_workspace_size(dtype, tokens, outs, width, dy, lddy,
                                                  ctypes.byref(any_)) == 0
    assert lib.b2g_linear_dweight8_workspace_size_ex(dtype, tokens, outs, width, dy, lddy, codes, ldq,
                                                     ctypes.byref(these)) == 0
    return any_.value, these.value


def test_arguments(lib):
    q, n = lib.b2g_linear_dweight8_workspace_size_ex, ctypes.c_size_t(99)
    assert q(5, 4, 8, 8, P, 8, P, 16, ctypes.byref(n)) == -12 and q(0, 4, 8, 8, P, 8, P, 16, None) == -3
    assert q(0, 4, 8, -8, P, 8, P, 16, ctypes.byref(n)) == -1
    for dims in ((0, 8, 8), (4, 0, 8), (4, 8, 0)):
        assert q(1, *dims, P, 8, P, 16, ctypes.byref(n)) == 0 and n.value == 0


# sizes whose x is read from its codes
CODES = [(300, 512, 256), (64, 4096, 4096), (5844, 128, 6944), (1, 8, 16), (20001, 64, 200)]


@pytest.mark.parametrize("tokens,outs,width", CODES)
def test_no_copy_of_x(lib, tokens, outs, width):
    """Codes on 16-byte boundaries need room for sums alone; others for x's copy in BF16 too."""
    copy = tokens * -(-width // 64) * 64 * 2
    most, these = asked(lib, 1, tokens, outs, width)
    # either way may leave sums, two for each piece of a tile of 256 rows; the copy is beside them
    sums = 2 * 256 * (256 if width > 128 else 128) * 4
    assert these % sums == 0 and these <= 2 * 76 * sums and most >= copy
    for other in (dict(codes=P + 8), dict(ldq=-(-width // 16) * 16 + 8)):
        assert copy <= asked(lib, 1, tokens, outs, width, **other)[1] <= most
    # FP32 dy: x is always prepared
    any_, these = asked(lib, 0, tokens, outs, width)
    assert any_ == these >= copy


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,outs,width", CODES + [(4096, 520, 2500), (1000, 1025, 777)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("codes_off", [0, 1])
def test_just_the_bytes_named(lib, tokens, outs, width, codes_off, dtype):
    """The C call with a workspace of that size between guards; one byte less is refused."""
    import dense_fp32_gemm_07_gb300 as b2g

    torch.manual_seed(tokens)
    ld, ldy = -(-width // 16) * 16, -(-outs // 8) * 8
    dy = torch.randn(tokens, ldy, device="cuda").to(dtype)[:, :outs]
    q, s = b2g.quantize_8bit(torch.randn(tokens, width, device="cuda"))
    room = torch.zeros(tokens * ld + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes = room.as_strided((tokens, width), (ld, 1), codes_off)
    codes.copy_(q)
    want = b2g.linear_weight_grad_8bit(dy, codes, s)
    code = 0 if dtype is torch.float32 else 1
    n = asked(lib, code, tokens, outs, width, dy.data_ptr(), ldy, codes.data_ptr(), ld)[1]
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    dw = torch.zeros_like(want)
    args = (code, tokens, outs, width, dy.data_ptr(), ldy, codes.data_ptr(), ld, s.data_ptr(), s.stride(0), 0,
            dw.data_ptr(), width)
    st = torch.cuda.current_stream().cuda_stream
    if n:
        assert lib.b2g_linear_dweight8(*args, ws.data_ptr(), n - 1, st) == b2g.B2G_ERR_WORKSPACE
        assert lib.b2g_linear_dweight8(*args, None, n, st) == b2g.B2G_ERR_WORKSPACE
    assert lib.b2g_linear_dweight8(*args, ws.data_ptr() if n else None, n, st) == 0
    torch.cuda.synchronize()
    assert torch.equal(dw, want) and (ws[n:] == 0xA5).all()
