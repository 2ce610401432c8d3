"""Argument checks of the 8-bit floating-point entry points and the balance loss (no GPU needed).

Every call below has at least one invalid argument, so it is refused before any HIP call;
pointers are never dereferenced. The Python functions' own checks run on CPU tensors.
"""
import ctypes

import pytest

import bit_gemm_token_amd as bgt

torch = pytest.importorskip("torch")

P = ctypes.c_void_p
OK, ODD2, ODD4, MIS16 = P(0x10000), P(0x10001), P(0x10002), P(0x10004)


@pytest.fixture(scope="module")
def L():
    return bgt.lib()


def refusals(call, pointers, types, shapes, mis16=()):
    """call(**changes) with NULL or misaligned pointers, unknown types and bad sizes."""
    for name in pointers:
        assert call(**{name: None}) == bgt.BGT_ERR_NULL, name
    for name in mis16:
        assert call(**{name: MIS16}) == bgt.BGT_ERR_ALIGN, name
    for name in types:
        for bad in (-1, 3):
            assert call(**{name: bad}) == bgt.BGT_ERR_MODE, name
    for bad in shapes:
        assert call(**bad) == bgt.BGT_ERR_SHAPE, bad


ROWS = [dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(K=0), dict(K=(1 << 18) + 1, ld=1 << 19)]


def test_rows(L):
    def quantize(x=OK, t=2, M=4, K=300, ld=300, q=OK, s=OK):
        return L.bgt_quantize_fp8(x, t, M, K, ld, q, s, None)

    def values(q=OK, s=OK, M=4, K=300, y=OK, t=2, ld=None):
        return L.bgt_dequantize_fp8(q, s, M, K, y, t, None)

    refusals(quantize, ("x", "q", "s"), ("t",), ROWS + [dict(ld=299)], ("q",))
    refusals(values, ("q", "s", "y"), ("t",), ROWS, ("q",))
    assert quantize(x=ODD2) == bgt.BGT_ERR_ALIGN and quantize(x=ODD4, t=0) == bgt.BGT_ERR_ALIGN
    assert values(y=ODD2) == bgt.BGT_ERR_ALIGN and values(y=ODD4, t=0) == bgt.BGT_ERR_ALIGN
    # more workgroups than a grid holds
    assert quantize(M=1 << 24, K=1 << 18, ld=1 << 18) == bgt.BGT_ERR_SHAPE


def test_weights(L):
    def pack(w=OK, t=0, E=2, K=256, N=64, qw=OK, sw=OK, qt=OK, st=OK):
        return L.bgt_pack_weights_fp8(w, t, E, K, N, qw, sw, qt, st, None)

    refusals(pack, ("w", "qw", "sw", "qt", "st"), ("t",),
             [dict(E=0), dict(E=257), dict(K=0), dict(N=0), dict(K=(1 << 18) + 1), dict(N=(1 << 18) + 1)], ("qw", "qt"))
    assert pack(w=ODD4) == bgt.BGT_ERR_ALIGN


def test_products(L):
    def gemm(qx=OK, sx=OK, qw=OK, sw=OK, M=4, N=64, K=256, y=OK, t=2, ld=None):
        return L.bgt_w8a8_gemm_fp8(qx, sx, qw, sw, M, N, K, y, t, None)

    def linear(x=OK, xt=2, ld=256, qw=OK, sw=OK, M=4, N=64, K=256, qx=OK, sx=OK, y=OK, t=2):
        return L.bgt_w8a8_linear_fp8(x, xt, ld, qw, sw, M, N, K, qx, sx, y, t, None)

    def moe(qx=OK, sx=OK, T=8, offs=OK, tok=OK, E=4, R=16, qw=OK, sw=OK, N=64, K=256, y=OK, t=2):
        return L.bgt_w8a8_moe_gemm_fp8(qx, sx, T, offs, tok, E, R, qw, sw, N, K, y, t, None)

    widths = [dict(N=0), dict(N=(1 << 18) + 1)]
    refusals(gemm, ("qx", "sx", "qw", "sw", "y"), ("t",), ROWS + widths, ("qx", "qw"))
    refusals(linear, ("x", "qw", "sw", "qx", "sx", "y"), ("xt", "t"), ROWS + widths + [dict(ld=255)], ("qx", "qw"))
    refusals(moe, ("qx", "sx", "offs", "tok", "qw", "sw", "y"), ("t",),
             widths + [dict(T=0), dict(T=(1 << 24) + 1), dict(E=0), dict(E=257), dict(R=0), dict(R=33), dict(K=0)], ("qx", "qw"))
    assert moe(offs=ODD4) == bgt.BGT_ERR_ALIGN and moe(tok=ODD4) == bgt.BGT_ERR_ALIGN
    for f in (gemm, linear, moe):
        assert f(y=ODD2) == bgt.BGT_ERR_ALIGN and f(y=ODD4, t=0) == bgt.BGT_ERR_ALIGN
    assert linear(x=ODD2) == bgt.BGT_ERR_ALIGN and linear(x=ODD4, xt=0) == bgt.BGT_ERR_ALIGN


def test_weight_gradients(L):
    def dense(qx=OK, sx=OK, dy=OK, t=2, ld=64, M=4, K=256, N=64, dw=OK, ws=OK, n=1 << 40):
        return L.bgt_wgrad_fp8(qx, sx, dy, t, ld, M, K, N, dw, ws, n, None)

    def moe(qx=OK, sx=OK, T=8, offs=OK, tok=OK, E=4, R=16, dy=OK, t=2, ld=64, K=256, N=64, dw=OK):
        return L.bgt_moe_wgrad_fp8(qx, sx, T, offs, tok, E, R, dy, t, ld, K, N, dw, None)

    shapes = [dict(N=0, ld=1), dict(N=(1 << 18) + 1, ld=1 << 19), dict(ld=63), dict(K=0), dict(K=(1 << 18) + 1)]
    refusals(dense, ("qx", "sx", "dy", "dw"), ("t",), shapes + [dict(M=0), dict(M=(1 << 24) + 1)], ("qx",))
    refusals(moe, ("qx", "sx", "offs", "tok", "dy", "dw"), ("t",),
             shapes + [dict(T=0), dict(E=0), dict(E=257), dict(R=0), dict(R=33)], ("qx",))
    for f in (dense, moe):
        assert f(dy=ODD2) == bgt.BGT_ERR_ALIGN and f(dw=ODD4, t=0) == bgt.BGT_ERR_ALIGN
    assert moe(offs=ODD4) == bgt.BGT_ERR_ALIGN and moe(tok=ODD4) == bgt.BGT_ERR_ALIGN
    for M, K, N in ((0, 256, 64), (4, 0, 64), (4, 256, 0)):
        assert L.bgt_wgrad_fp8_workspace_bytes(M, K, N) == bgt.BGT_ERR_SHAPE
    for M, K, N in ((1, 1, 1), (8192, 256, 256), (1 << 20, 4096, 4096), (100000, 300, 1000)):
        need = L.bgt_wgrad_fp8_workspace_bytes(M, K, N)
        assert need >= 0 and need % 4 == 0
        if need:
            assert dense(M=M, K=K, N=N, ld=N, ws=None, n=need) == bgt.BGT_ERR_NULL
            assert dense(M=M, K=K, N=N, ld=N, n=need - 1) == bgt.BGT_ERR_SHAPE
            assert dense(M=M, K=K, N=N, ld=N, ws=ODD4, n=need) == bgt.BGT_ERR_ALIGN


def test_gate(L):
    def gate(g=OK, ld=300, u=OK, ldu=300, t=2, M=4, K=300, hq=OK, hs=OK, gq=OK, gs=OK, uq=OK, us=OK):
        return L.bgt_silu_mul_fp8(g, ld, u, ldu, t, M, K, hq, hs, gq, gs, uq, us, None)

    def grad(dh=OK, t=2, ld=300, gq=OK, gs=OK, uq=OK, us=OK, M=4, K=300, dg=OK, du=OK):
        return L.bgt_silu_mul_fp8_backward(dh, t, ld, gq, gs, uq, us, M, K, dg, du, None)

    refusals(gate, ("g", "u", "hq", "hs", "gq", "gs", "uq", "us"), ("t",), ROWS + [dict(ld=299), dict(ldu=299)], ("hq", "gq", "uq"))
    refusals(grad, ("dh", "gq", "gs", "uq", "us", "dg", "du"), ("t",), ROWS + [dict(ld=299)], ("gq", "uq"))
    for name in ("g", "u"):
        assert gate(**{name: ODD2}) == bgt.BGT_ERR_ALIGN
    for name in ("dh", "dg", "du"):
        assert grad(**{name: ODD2}) == bgt.BGT_ERR_ALIGN


def test_balance(L):
    def loss(l=OK, t=0, ld=8, ids=OK, T=4, E=8, k=2, loss=OK, c=OK, p=OK, n=OK, ws=OK, size=1 << 30):  # noqa: E741
        return L.bgt_moe_balance(l, t, ld, ids, T, E, k, loss, c, p, n, ws, size, None)

    def grad(d=OK, l=OK, t=0, ld=8, c=OK, n=OK, T=4, E=8, out=OK):  # noqa: E741
        return L.bgt_moe_balance_backward(d, l, t, ld, c, n, T, E, out, None)

    sizes = [dict(T=0), dict(T=(1 << 24) + 1), dict(E=0), dict(E=257, ld=257), dict(ld=7)]
    refusals(loss, ("l", "ids", "loss", "c", "p", "n", "ws"), ("t",), sizes + [dict(k=0), dict(k=9), dict(k=17, E=32, ld=32)])
    refusals(grad, ("d", "l", "c", "n", "out"), ("t",), sizes)
    for name in ("l", "ids", "loss", "c", "p", "n", "ws"):
        assert loss(**{name: ODD4}) == bgt.BGT_ERR_ALIGN
    for name in ("d", "l", "c", "n", "out"):
        assert grad(**{name: ODD4}) == bgt.BGT_ERR_ALIGN
    for T, E in ((1, 1), (61, 8), (16381, 64), (1 << 24, 256)):
        need = L.bgt_moe_balance_workspace_bytes(T, E)
        assert need > 0 and need % 4 == 0
        assert loss(T=T, E=E, ld=E, k=1, size=need - 1) == bgt.BGT_ERR_SHAPE
    assert L.bgt_moe_balance_workspace_bytes(0, 8) == bgt.BGT_ERR_SHAPE


def test_python_checks():
    """Tensors off the GPU, of other shapes and dtypes are refused before the library is called."""
    x = torch.zeros(4, 256)
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 4, dtype=torch.float8_e8m0fnu)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: bgt.quantize_fp8(x), lambda: bgt.dequantize_fp8(q, s), lambda: bgt.pack_weights_fp8(x),
                 lambda: bgt.w8a8_gemm_fp8(q, s, q, s), lambda: bgt.w8a8_linear_fp8(x, q, s),
                 lambda: bgt.w8a8_moe_gemm_fp8(q, s, ids, ids, q, s), lambda: bgt.wgrad_fp8(q, s, x),
                 lambda: bgt.moe_wgrad_fp8(q, s, ids, ids, x), lambda: bgt.silu_mul_fp8(x, x),
                 lambda: bgt.silu_mul_fp8_backward(x, q, s, q, s), lambda: bgt.moe_balance(x, ids),
                 lambda: bgt.moe_balance_backward(x, x, ids, ids), lambda: bgt.quantize_fp8([1.0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        bgt.pack_weights_fp8(torch.zeros(4))
    for K in (0, 128, 257):
        with pytest.raises(ValueError):
            bgt._logical(K, 256)
    assert bgt._logical(129, 256) == 129 and bgt._logical(None, 256) == 256
