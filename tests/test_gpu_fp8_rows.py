"""Rows and weights in 8-bit floating point, the gated activation and its gradient, against 64 bits.

Codes, exponents and values are exact: x / 2^e is exact in fp32 and rounded once, so they are
compared for equality. The gated activation is computed in fp32 first.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp8_plain as plain  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def bgt():
    import bit_gemm_token_amd
    bit_gemm_token_amd.lib()
    return bit_gemm_token_amd


def some_rows(seed, M, K, dev, dtype):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=dev) * torch.exp2(torch.randint(-12, 6, (M, 1), generator=g, device=dev).float())
    x[:, ::37] *= 20
    if M > 2:
        x[1] = 0                                        # blocks of zeros
        x[2, :K // 2] = 0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (17, 129), (64, 4096), (65, 1000), (1021, 264), (4096, 1408)])
def test_rows(bgt, dev, dtype, M, K):
    x = some_rows(M + K, M, K, dev, dtype)
    q, s = bgt.quantize_fp8(x)
    codes, e = plain.rows(x)
    assert torch.equal(plain.exponents_of(s), e)
    assert torch.equal(q.double(), codes)
    for out in TYPES:
        y = bgt.dequantize_fp8(q, s, K, out_dtype=out)
        assert torch.equal(y, (codes.view(M, -1, 128) * torch.exp2(e.t())[..., None]).view(M, -1)[:, :K].to(out))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_strides(bgt, dev, dtype):
    big = some_rows(5, 40, 700, dev, dtype)
    for x in (big[:, :640], big[:, 8:648], big[:, 1:300], big[::3, 16:272], big[7:8, 3:200]):
        q, s = bgt.quantize_fp8(x)
        codes, e = plain.rows(x)
        assert torch.equal(plain.exponents_of(s), e) and torch.equal(q.double(), codes)
    q, s = bgt.quantize_fp8(big)
    y = torch.empty(40 * 700 + 1, device=dev, dtype=dtype)[1:].view(40, 700)   # misaligned output
    assert torch.equal(bgt.dequantize_fp8(q, s, y=y, K=700), bgt.dequantize_fp8(q, s, K=700, out_dtype=dtype))


def test_range_and_ties(bgt, dev):
    """Every power of two a block may hold, values at 448 * 2^e and next to it, ties, the type's
    largest, subnormals; and blocks that are not finite."""
    tops = torch.exp2(torch.arange(-149, 128, device=dev, dtype=torch.float64)).float()
    x = torch.zeros(tops.numel() * 3, 128, device=dev)
    x[:, 0] = torch.cat([tops, tops * 1.75, torch.nextafter(tops * 1.75, torch.tensor(1e39, device=dev))])
    x[:, 1:] = x[:, :1] * torch.linspace(-1, 1, 127, device=dev)
    x = x[torch.isfinite(x).all(1)]
    q, s = bgt.quantize_fp8(x)
    codes, e = plain.rows(x)
    assert torch.equal(plain.exponents_of(s), e) and torch.equal(q.double(), codes)
    half = torch.arange(-448 * 512, 448 * 512 + 1, 1, device=dev, dtype=torch.float64) / 1024      # steps of 2^-10
    x = torch.cat([half, half.new_zeros(-half.numel() % 127)]).view(-1, 127)
    x = torch.cat([torch.full_like(x[:, :1], 448.0), x], 1).float()                                # e = 0
    q, s = bgt.quantize_fp8(x)
    assert bool((plain.exponents_of(s) == 0).all()) and torch.equal(q.double(), plain.e4m3(x.double()))
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.ones(3, 256, device=dev)
        x[1, 130] = bad
        q, s = bgt.quantize_fp8(x)
        assert s.view(torch.uint8).tolist() == [[119] * 3, [119, 255, 119]]
        y = bgt.dequantize_fp8(q, s)
        assert bool(y[1, 128:].isnan().all()) and torch.equal(y[::2], x[::2]) and torch.equal(y[1, :128], x[1, :128])


def test_every_code_and_exponent(bgt, dev):
    q = torch.arange(256, dtype=torch.uint8, device=dev).view(2, 128).view(torch.float8_e4m3fn)
    for b in range(0, 256, 5):
        s = torch.full((1, 2), b, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
        y = bgt.dequantize_fp8(q, s)
        assert plain.same(y, (q.double() * s.double().view(2, 1)).float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,K,N", [(None, 128, 128), (None, 1, 1), (None, 300, 200), (None, 4096, 1408), (3, 129, 257), (2, 256, 24)])
def test_weights(bgt, dev, dtype, E, K, N):
    g = torch.Generator(device=dev).manual_seed(K + N)
    w = (0.02 * torch.randn(E or 1, K, N, generator=g, device=dev)).to(dtype)
    w[:, : K // 3] *= 30
    p = bgt.pack_weights_fp8(w if E else w[0], turned=True)
    one = bgt.pack_weights_fp8(w if E else w[0])
    for name in ("qw", "sw"):
        assert torch.equal(one[name].view(torch.uint8), p[name].view(torch.uint8))
    for e in range(E or 1):
        codes, ex = plain.weights(w[e])
        at = (lambda t: t[e]) if E else (lambda t: t)
        assert torch.equal(plain.exponents_of(at(p["sw"])), ex)
        assert torch.equal(plain.exponents_of(at(p["st"])), ex.t())
        assert torch.equal(at(p["qw"]).double(), codes.t()[:N])
        assert torch.equal(at(p["qt"]).double(), codes[:K])


def gate_rows(seed, M, K, dev, dtype):
    g = torch.Generator(device=dev).manual_seed(seed)
    return [(4 * torch.randn(M, K, generator=g, device=dev)).to(dtype) for _ in range(3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (33, 127), (70, 1000), (515, 1408), (2048, 2048)])
def test_gate(bgt, dev, dtype, M, K):
    g, u, _ = gate_rows(M * K, M, K, dev, dtype)
    hq, hs, gq, gs, uq, us = bgt.silu_mul_fp8(g, u)
    for x, q, s in ((g, gq, gs), (u, uq, us)):
        codes, e = plain.rows(x)
        assert torch.equal(plain.exponents_of(s), e) and torch.equal(q.double(), codes)
    h = torch.nn.functional.silu(g.double()) * u.double()
    # h in fp32 is off by a few roundings (2^-20 of itself is 16), which may move a block's
    # largest across a power of two's border, and then half a step of the code
    top, e = plain.blocks(h).abs().amax(2), plain.exponents_of(hs).t()
    assert bool((top <= 448 * torch.exp2(e) * (1 + 2.0 ** -20)).all())
    assert bool(((top > 224 * torch.exp2(e) * (1 - 2.0 ** -20)) | (e == plain.LOW)).all())
    step = torch.maximum(2.0 ** -4 * plain.blocks(h).abs(), 2.0 ** -10 * torch.exp2(e)[..., None])
    off = (plain.values(hq, hs).view(step.shape) - plain.blocks(h)).abs()
    assert bool((off <= step * (1 + 2.0 ** -18) + 2.0 ** -20 * plain.blocks(h).abs()).all())


def gate_gradients(g, u, dh):
    s = torch.sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def check_gate_gradients(out, g, u, dh):
    dtype, s = out[0].dtype, torch.sigmoid(g)
    dg, du = gate_gradients(g, u, dh)
    # fp32: 1 - s is off by 2^-24, times |g|; exp, division and products by a few 2^-24 each
    size = (dh * u).abs() * s * (1 + g.abs())
    half = torch.finfo(dtype).eps / 2
    assert bool(((out[0].double() - dg).abs() <= 16 * 2.0 ** -24 * size + half * dg.abs() * 1.01 + plain.smallest(dtype) + 1e-36 * size).all())
    assert bool(((out[1].double() - du).abs() <= 16 * 2.0 ** -24 * du.abs() + half * du.abs() * 1.01 + plain.smallest(dtype)).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (33, 127), (70, 1000), (515, 1408), (2048, 2048)])
def test_gate_gradient(bgt, dev, dtype, M, K):
    g, u, dh = gate_rows(M * K + 1, M, K, dev, dtype)
    _, _, gq, gs, uq, us = bgt.silu_mul_fp8(g, u)
    out = bgt.silu_mul_fp8_backward(dh, gq, gs, uq, us)
    check_gate_gradients(out, plain.values(gq, gs)[:, :K], plain.values(uq, us)[:, :K], dh.double())


@pytest.mark.parametrize("dtype", TYPES)
def test_gate_of_strides(bgt, dev, dtype):
    """gate and up as the halves of one matrix, rows of dh apart."""
    both = torch.cat(gate_rows(9, 50, 384, dev, dtype)[:2], 1)
    a = bgt.silu_mul_fp8(both[:, :384], both[:, 384:])
    b = bgt.silu_mul_fp8(both[:, :384].contiguous(), both[:, 384:].contiguous())
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    dh = gate_rows(10, 50, 400, dev, dtype)[0]
    for part in (dh[:, :384], dh[:, 3:387]):
        x, y = bgt.silu_mul_fp8_backward(part, *b[2:]), bgt.silu_mul_fp8_backward(part.contiguous(), *b[2:])
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_gate_gradient_is_the_difference(bgt, dev):
    """Against central differences, in 64 bits, of silu(g) * u at the kept values."""
    g, u, dh = gate_rows(11, 20, 256, dev, torch.float32)
    _, _, gq, gs, uq, us = bgt.silu_mul_fp8(g, u)
    dg, du = bgt.silu_mul_fp8_backward(dh, gq, gs, uq, us)
    gv, uv, d = plain.values(gq, gs), plain.values(uq, us), 1e-5
    h = lambda a, b: torch.nn.functional.silu(a) * b  # noqa: E731
    dh = dh.double()
    # the difference's own error: d^2 of third derivatives (below 1) and 2^-53 / d
    size = dh.abs() * (1 + uv.abs()) * (1 + gv.abs())
    assert bool(((h(gv + d, uv) - h(gv - d, uv)) / (2 * d) * dh - dg.double()).abs().le(2e-6 * size).all())
    assert bool(((h(gv, uv + d) - h(gv, uv - d)) / (2 * d) * dh - du.double()).abs().le(2e-6 * size).all())


def test_gate_extremes(bgt, dev):
    """Large gates of both signs: silu goes to g and to 0, its slope to 1 and to 0."""
    g = torch.tensor([[-1e30, -200.0, -89.0, -20.0, 0.0, 20.0, 200.0, 1e30]], device=dev).repeat(1, 16)
    u = torch.full_like(g, 0.5)
    hq, hs, gq, gs, uq, us = bgt.silu_mul_fp8(g, u)
    h = bgt.dequantize_fp8(hq, hs)
    assert bool(h.isfinite().all()) and float(h[0, 7]) == pytest.approx(5e29, rel=2.0 ** -4) and float(h[0, 0]) == 0
    dh = torch.ones_like(g)
    dg, du = bgt.silu_mul_fp8_backward(dh, *bgt.quantize_fp8(g.clamp(-400, 400)), uq, us)
    gv = bgt.dequantize_fp8(*bgt.quantize_fp8(g.clamp(-400, 400))).double()
    check_gate_gradients((dg, du), gv, u.double(), dh.double())


def test_many_elements(bgt, dev):
    """Offsets past 2^31."""
    M, K = (1 << 18) + 5, 8192
    x = torch.zeros(M, K, device=dev, dtype=torch.bfloat16)
    g = torch.Generator(device=dev).manual_seed(1)
    x[-40:] = torch.randn(40, K, generator=g, device=dev).to(torch.bfloat16)
    q, s = bgt.quantize_fp8(x)
    codes, e = plain.rows(x[-40:])
    assert torch.equal(q[-40:].double(), codes) and torch.equal(plain.exponents_of(s[:, -40:]), e)
    assert not bool(q[:-40].view(torch.uint8).any())
    y = bgt.dequantize_fp8(q, s, out_dtype=torch.bfloat16)
    assert torch.equal(y[-40:], (codes.view(40, -1, 128) * torch.exp2(e.t())[..., None]).view(40, -1).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_gate_not_finite(bgt, dev, dtype, which, bad):
    """What is not finite in gate or up makes its block of that and of the product NaN, no other."""
    rows = gate_rows(12, 9, 300, dev, dtype)[:2]
    clean = bgt.silu_mul_fp8(*rows)
    rows[which][4, 140] = bad
    out = bgt.silu_mul_fp8(*rows)
    for i in range(3):                                        # h, gate, up
        v, c = bgt.dequantize_fp8(*out[2 * i:2 * i + 2]), bgt.dequantize_fp8(*clean[2 * i:2 * i + 2])
        if i in (0, 1 + which):
            assert bool(v[4, 128:256].isnan().all())
            v[4, 128:256] = c[4, 128:256]
        assert torch.equal(v, c)


def test_gate_at_the_ends_of_fp32(bgt, dev):
    """Gates up to the largest fp32 value, and products that pass it."""
    top = torch.finfo(torch.float32).max
    g = torch.tensor([-top, top, -3e38, 2.5e38, -87.0, 87.0, -104.0, 104.0], device=dev).repeat(16)[None]
    h = plain.values(*bgt.silu_mul_fp8(g, torch.ones_like(g))[:2])   # top rounds to 2^128, past fp32
    ref = torch.nn.functional.silu(g.double())
    # codes of 2^-4, on a block whose largest is top: below 2^-9 of 2^e = top / 448 they are 0
    assert bool(((h - ref).abs() <= 2.0 ** -4 * ref.abs() + 2.0 ** -10 * 2.0 ** 120).all())
    over = bgt.dequantize_fp8(*bgt.silu_mul_fp8(g, torch.full_like(g, 4.0))[:2])
    assert bool(over.isnan().all())                           # an infinity in the block
