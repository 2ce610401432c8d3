"""A weight's gradient from rows kept in 8 bits, of one matrix and of every expert, against 64 bits.

Products are exact (the kept values in bf16, dy in one to three bf16 terms), sums fp32: within
the number of terms times 2^-23 of the sum of magnitudes, and of the norm within the rounding
of the output and a random walk of such roundings.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp8_plain as plain  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
TERMS = {torch.float32: 3, torch.float16: 2, torch.bfloat16: 1}


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


def inputs(seed, T, R, K, N, dev, dtype):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=dev) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g, device=dev).float())
    dy = torch.randn(R, N, generator=g, device=dev) * torch.exp2(torch.randint(-3, 3, (R, 1), generator=g, device=dev).float())
    return x, dy.to(dtype)


def check(dw, x, dy):
    """dw against x^T dy (x doubles)."""
    dtype, M = dw.dtype, max(1, x.shape[0])
    ref, size = x.t() @ dy.double(), x.abs().t() @ dy.double().abs()
    half, n = torch.finfo(dtype).eps / 2, TERMS[dtype] * M
    bound = n * 2.0 ** -23 * size + half * (1 + n * 2.0 ** -23) * ref.abs() + plain.smallest(dtype)
    assert bool(((dw.double() - ref).abs() <= bound).all()), float(((dw.double() - ref).abs() / bound.clamp(min=1e-300)).max())
    assert plain.rel(dw, ref) <= half + 8 * 2.0 ** -24 * n ** 0.5


SHAPES = [(1, 1, 1), (1, 128, 256), (5, 130, 77), (31, 300, 256), (32, 256, 257), (33, 1000, 130), (64, 513, 512), (100, 128, 128),
          (257, 384, 640), (1000, 256, 256), (1021, 272, 258), (4096, 512, 300), (3000, 1408, 1024),
          (600, 3000, 4200), (600, 3000, 4203), (130, 3000, 4200), (300, 256, 3), (2100, 130, 7), (2500, 130, 77), (520, 4100, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_dense(bgt, dev, dtype, M, K, N):
    print("wgrad", M, K, N, dtype, flush=True)
    x, dy = inputs(M + K + N, M, M, K, N, dev, dtype)
    q, s = bgt.quantize_fp8(x)
    dw = bgt.wgrad_fp8(q, s, dy, K, dw=torch.full((K, N), float("nan"), device=dev, dtype=dtype))
    check(dw, plain.values(q, s)[:, :K], dy)
    assert torch.equal(dw, bgt.wgrad_fp8(q, s, dy, K))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(bgt, dev, dtype):
    x, dy = inputs(2, 90, 90, 256, 400, dev, dtype)
    q, s = bgt.quantize_fp8(x)
    for part in (dy[:, :256], dy[:, 1:258], dy[:, 3:6], dy[:, 2:100]):
        dw = bgt.wgrad_fp8(q, s, part)
        check(dw, plain.values(q, s), part)
        assert torch.equal(dw, bgt.wgrad_fp8(q, s, part.contiguous()))


ROUTED = [(1, 8, 2, 0.0, 128, 256), (7, 4, 1, 0.3, 130, 77), (61, 8, 2, 0.0, 512, 256), (300, 5, 3, 0.2, 256, 300),
          (1000, 32, 4, 0.1, 264, 128), (9, 4, 2, 1.0, 256, 64), (700, 2, 2, 0.0, 384, 129),
          (1100, 2, 1, 0.0, 2600, 2600), (1200, 2, 1, 0.1, 2600, 2601), (50, 4, 2, 0.1, 130, 5), (900, 32, 4, 0.1, 1024, 264)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,drop,K,N", ROUTED)
def test_routed(bgt, dev, dtype, T, E, k, drop, K, N):
    print("routed wgrad", T, E, k, K, N, dtype, flush=True)
    x, dy = inputs(T + K + N, T, T * k, K, N, dev, dtype)
    g = torch.Generator(device=dev).manual_seed(T)
    offs, tok, expert = plain.route(plain.ids_of(g, T, E, k, drop, dev), E)
    dy[len(expert):] = float("nan")                           # rows without a slot are not read
    q, s = bgt.quantize_fp8(x)
    dw = bgt.moe_wgrad_fp8(q, s, offs, tok, dy, K, dw=torch.full((E, K, N), float("nan"), device=dev, dtype=dtype))
    v = plain.values(q, s)[:, :K]
    for e in range(E):
        a, b = int(offs[e]), int(offs[e + 1])
        check(dw[e], v[tok[a:b].long()], dy[a:b])


def test_two_streams(bgt, dev):
    """Equal bits on two streams at once, with workspaces (parts of the rows) and without."""
    cases = []
    for M, K, N in ((4096, 256, 264), (700, 1024, 512), (61, 512, 77)):
        x, dy = inputs(M, M, M, K, N, dev, torch.bfloat16)
        cases.append((*bgt.quantize_fp8(x), dy))
    ref = [bgt.wgrad_fp8(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append([bgt.wgrad_fp8(*c) for c in cases])
        torch.cuda.synchronize()
        for out in got:
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_gradient_of_the_product(bgt, dev):
    """dW is the difference, in 64 bits, of sum(dy * (x8 W)) in W: linear, so exact but for roundings."""
    x, dy = inputs(8, 50, 50, 128, 40, dev, torch.float32)
    q, s = bgt.quantize_fp8(x)
    dw, v = bgt.wgrad_fp8(q, s, dy), plain.values(q, s)
    g = torch.Generator(device=dev).manual_seed(1)
    for _ in range(5):
        d = torch.randn(128, 40, generator=g, device=dev).double()
        w = torch.randn(128, 40, generator=g, device=dev).double()
        f = lambda m: ((v @ m) * dy.double()).sum()  # noqa: E731
        assert float((dw.double() * d).sum()) == pytest.approx(float(f(w + d) - f(w - d)) / 2, rel=1e-5, abs=1e-4 * float(v.abs().sum()))


@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite(bgt, dev, dtype):
    """An infinity in dy reaches its column, one in a kept block the block's 128 rows, as the
    formula lets them."""
    x, dy = inputs(4, 70, 70, 300, 50, dev, dtype)
    q, s = bgt.quantize_fp8(x)
    clean = bgt.wgrad_fp8(q, s, dy, 300)
    dy[40, 7] = float("inf")
    dw = bgt.wgrad_fp8(q, s, dy, 300)
    want = plain.values(q, s)[40, :300] * float("inf")        # NaN where the kept value is 0
    assert plain.same(dw[:, 7].double(), want)
    dw[:, 7] = clean[:, 7]
    assert torch.equal(dw, clean)
    dy[40, 7] = float("nan")
    assert bool(bgt.wgrad_fp8(q, s, dy, 300)[:, 7].isnan().all())
    dy[40, 7] = 0
    x[3, 130] = float("inf")
    dw = bgt.wgrad_fp8(*bgt.quantize_fp8(x), dy, 300)
    assert bool(dw[128:256].isnan().all()) and not bool(dw[:128].isnan().any()) and not bool(dw[256:].isnan().any())


@pytest.mark.parametrize("N", [5, 50, 56])
@pytest.mark.parametrize("dtype", TYPES)
def test_last_row_not_finite(bgt, dev, dtype, N):
    """What fills up the last step of the rows takes nothing from the last row."""
    x, dy = inputs(N, 67, 67, 256, N, dev, dtype)
    dy[66, 1], dy[66, 3] = float("inf"), float("nan")
    q, s = bgt.quantize_fp8(x)
    dw = bgt.wgrad_fp8(q, s, dy)
    assert plain.same(dw[:, 1].double(), plain.values(q, s)[66] * float("inf")) and bool(dw[:, 3].isnan().all())
    rest = [n for n in range(N) if n not in (1, 3)]
    check(dw[:, rest], plain.values(q, s), dy[:, rest])


def test_many_elements(bgt, dev):
    """Codes and dy past 2^31 bytes."""
    M, K, N = (1 << 18) + 70, 8192, 64
    q = torch.zeros(M, K, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.full((K // 128, M), 127, device=dev, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    x, dy = inputs(3, 80, 80, K, N, dev, torch.bfloat16)
    a, b = bgt.quantize_fp8(x)
    q[-80:].view(torch.uint8).copy_(a.view(torch.uint8))
    s.view(torch.uint8)[:, -80:].copy_(b.view(torch.uint8))
    wide = torch.zeros(M, 16384, device=dev, dtype=torch.bfloat16)
    wide[-80:, :N] = dy
    check(bgt.wgrad_fp8(q, s, wide[:, :N]), plain.values(a, b), dy)
