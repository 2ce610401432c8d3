"""Argument checks of the routing, row and weight-only entry points (no GPU needed).

Every call below has at least one invalid argument, so it is refused before any
HIP call; pointers are never dereferenced.
"""
import ctypes

import pytest

import bit_gemm_token_amd as bgt

P = ctypes.c_void_p
OK, ODD2, ODD4 = P(0x10000), P(0x10001), P(0x10002)     # aligned; off by 1; off by 2 bytes
MIS16 = P(0x10004)


@pytest.fixture(scope="module")
def L():
    return bgt.lib()


SHAPES = [(0, 8, 2), (4, 0, 1), (4, 257, 2), (4, 8, 0), (4, 8, 9), (4, 32, 17), ((1 << 24) + 1, 8, 1),
          ((1 << 23) + 1, 8, 2), (-1, 8, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_shapes(L, T, E, k):
    want = bgt.BGT_ERR_SHAPE
    assert L.bgt_moe_sort_workspace_bytes(T, E, k) == want
    assert L.bgt_moe_route(OK, 0, max(E, 1), T, E, k, 0, OK, OK, OK, OK, OK, OK, 1 << 40, None) == want
    assert L.bgt_moe_sort(OK, T, E, k, OK, OK, OK, OK, 1 << 40, None) == want
    assert L.bgt_moe_route_backward(OK, OK, 0, max(E, 1), OK, T, E, k, 0, OK, None) == want
    assert L.bgt_moe_gather(OK, 0, 64, OK, OK, T, E, k, 64, OK, None) == want
    assert L.bgt_moe_combine_backward(OK, 64, OK, 0, OK, OK, OK, T, E, k, 64, OK, OK, None) == want


def test_workspace_sizes(L):
    for T, E, k in ((1, 8, 2), (64, 256, 16), (4096, 8, 2), (1 << 20, 256, 16)):
        need = L.bgt_moe_sort_workspace_bytes(T, E, k)
        assert need >= 0 and need % 4 == 0
        if need:                                      # missing or too small
            assert L.bgt_moe_sort(OK, T, E, k, OK, OK, OK, None, need, None) == bgt.BGT_ERR_NULL
            assert L.bgt_moe_sort(OK, T, E, k, OK, OK, OK, OK, need - 1, None) == bgt.BGT_ERR_SHAPE
            assert L.bgt_moe_sort(OK, T, E, k, OK, OK, OK, ODD4, need, None) == bgt.BGT_ERR_ALIGN


def test_route(L):
    def call(logits=OK, type=0, ld=8, T=4, E=8, k=2, norm=0, w=OK, ids=OK, offs=OK, tok=OK, pos=OK):
        return L.bgt_moe_route(logits, type, ld, T, E, k, norm, w, ids, offs, tok, pos, OK, 1 << 40, None)

    for name in ("logits", "w", "ids", "offs", "tok", "pos"):
        assert call(**{name: None}) == bgt.BGT_ERR_NULL
        assert call(**{name: ODD4}) == bgt.BGT_ERR_ALIGN
    assert call(logits=ODD2, type=1) == bgt.BGT_ERR_ALIGN
    assert call(type=3) == bgt.BGT_ERR_MODE
    assert call(type=-1) == bgt.BGT_ERR_MODE
    assert call(norm=2) == bgt.BGT_ERR_MODE
    assert call(ld=7) == bgt.BGT_ERR_SHAPE


def test_route_backward(L):
    def call(dw=OK, logits=OK, type=0, ld=8, ids=OK, norm=0, out=OK):
        return L.bgt_moe_route_backward(dw, logits, type, ld, ids, 4, 8, 2, norm, out, None)

    for name in ("dw", "logits", "ids", "out"):
        assert call(**{name: None}) == bgt.BGT_ERR_NULL
        assert call(**{name: ODD4}) == bgt.BGT_ERR_ALIGN
    assert call(type=5) == bgt.BGT_ERR_MODE
    assert call(norm=-1) == bgt.BGT_ERR_MODE
    assert call(ld=0) == bgt.BGT_ERR_SHAPE


def test_rows(L):
    def gather(x=OK, type=2, ld=64, offs=OK, pos=OK, H=64, xs=OK):
        return L.bgt_moe_gather(x, type, ld, offs, pos, 4, 8, 2, H, xs, None)

    def combine(ys=OK, type=2, pos=OK, w=OK, H=64, y=OK, T=4, k=2):
        return L.bgt_moe_combine(ys, type, pos, w, T, k, H, y, None)

    def back(dy=OK, ld=64, ys=OK, type=2, offs=OK, pos=OK, w=OK, H=64, dys=OK, dw=OK):
        return L.bgt_moe_combine_backward(dy, ld, ys, type, offs, pos, w, 4, 8, 2, H, dys, dw, None)

    for name in ("x", "offs", "pos", "xs"):
        assert gather(**{name: None}) == bgt.BGT_ERR_NULL
        assert gather(**{name: ODD2}) == bgt.BGT_ERR_ALIGN
    for name in ("ys", "pos", "y"):
        assert combine(**{name: None}) == bgt.BGT_ERR_NULL
        assert combine(**{name: ODD2}) == bgt.BGT_ERR_ALIGN
    assert combine(w=ODD4) == bgt.BGT_ERR_ALIGN
    assert combine(T=0) == bgt.BGT_ERR_SHAPE and combine(k=17) == bgt.BGT_ERR_SHAPE
    for name in ("dy", "ys", "offs", "pos", "w", "dys", "dw"):
        assert back(**{name: None}) == bgt.BGT_ERR_NULL
        assert back(**{name: ODD2}) == bgt.BGT_ERR_ALIGN
    for f in (gather, combine, back):
        assert f(type=7) == bgt.BGT_ERR_MODE
        assert f(H=0) == bgt.BGT_ERR_SHAPE
        assert f(H=(1 << 20) + 1) == bgt.BGT_ERR_SHAPE
    assert gather(ld=63) == bgt.BGT_ERR_SHAPE and back(ld=63) == bgt.BGT_ERR_SHAPE


def test_w4a16(L):
    def gemv(x=OK, xt=2, ld=256, pk=OK, fs=OK, M=2, N=32, K=256, y=OK, yt=2):
        return L.bgt_w4a16_gemv(x, xt, ld, pk, fs, M, N, K, y, yt, None)

    def moe(x=OK, xt=2, ld=256, T=4, offs=OK, tok=OK, E=8, R=8, pk=OK, fs=OK, N=32, K=256, y=OK, yt=2):
        return L.bgt_w4a16_moe_gemv(x, xt, ld, T, offs, tok, E, R, pk, fs, N, K, y, yt, None)

    for f in (gemv, moe):
        for name in ("x", "pk", "fs", "y"):
            assert f(**{name: None}) == bgt.BGT_ERR_NULL
        for name in ("pk", "fs", "y"):
            assert f(**{name: MIS16}) == bgt.BGT_ERR_ALIGN
        assert f(x=ODD2) == bgt.BGT_ERR_ALIGN
        assert f(x=ODD4, xt=0) == bgt.BGT_ERR_ALIGN
        assert f(xt=3) == bgt.BGT_ERR_MODE and f(yt=-1) == bgt.BGT_ERR_MODE
        assert f(ld=255) == bgt.BGT_ERR_SHAPE
        for bad in (dict(N=0), dict(N=24), dict(N=(1 << 24) + 16), dict(K=0), dict(K=200, ld=200),
                    dict(K=65664, ld=65664)):
            assert f(**bad) == bgt.BGT_ERR_SHAPE
    assert gemv(M=0) == bgt.BGT_ERR_SHAPE and gemv(M=65537) == bgt.BGT_ERR_SHAPE
    for bad in (dict(T=0), dict(E=0), dict(E=257, R=1), dict(R=0), dict(R=33)):
        assert moe(**bad) == bgt.BGT_ERR_SHAPE
    for name in ("offs", "tok"):
        assert moe(**{name: None}) == bgt.BGT_ERR_NULL
        assert moe(**{name: ODD4}) == bgt.BGT_ERR_ALIGN
