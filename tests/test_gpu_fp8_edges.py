"""8-bit floating-point operators at the edges of their types' ranges, against 64 bits."""
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


def within(y, x, w, dtype):
    ref = x @ w
    bound = plain.product_bound(x, w, ref, dtype)
    assert bool(y.isfinite().all())
    assert bool(((y.double() - ref).abs() <= bound).all()), float(((y.double() - ref).abs() / bound).max())


# powers of two of x and w whose product is well within the types; fp16 holds sums of 256 products of
# 2^6 (at most 3.61 * 2^14 = 59146), and no more of them
FAR = [(118, -20), (-20, 118), (118, -112), (-112, 118), (127, -122), (-122, 127)]


@pytest.mark.parametrize("a,b", FAR)
@pytest.mark.parametrize("M,K", [(1, 128), (1, 256), (20, 256), (60, 256), (300, 256), (1, 4224), (20, 4224), (60, 4224)])
def test_products_of_far_scales(bgt, dev, M, K, a, b):
    """Neither factor's scale alone takes a sum out of range, whichever is the large one; groups of
    either sign."""
    N = 40
    g = torch.Generator(device=dev).manual_seed(M + K)
    x = (1 + 0.9 * torch.rand(M, K, generator=g, device=dev)) * 2.0 ** a
    w = (1 + 0.9 * torch.rand(K, N, generator=g, device=dev)) * 2.0 ** b
    x[:, 128:256] *= -0.5
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    for dtype in TYPES if a + b <= 6 and K <= 256 else TYPES[::2]:
        y = bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=dtype)
        within(y, plain.values(q, s), plain.matrix(p["qw"], p["sw"]), dtype)
        z = bgt.w8a8_linear_fp8(x, p["qw"], p["sw"], out_dtype=dtype)[0]
        within(z, plain.values(q, s), plain.matrix(p["qw"], p["sw"]), dtype)


@pytest.mark.parametrize("a,b", FAR)
@pytest.mark.parametrize("T,K", [(3, 256), (30, 256), (90, 256), (400, 256), (30, 4224)])
def test_routed_products_of_far_scales(bgt, dev, T, K, a, b):
    E, N = 2, 40
    g = torch.Generator(device=dev).manual_seed(T + K)
    x = (1 + 0.9 * torch.rand(T, K, generator=g, device=dev)) * 2.0 ** a
    w = (1 + 0.9 * torch.rand(E, K, N, generator=g, device=dev)) * 2.0 ** b
    x[:, 128:256] *= -0.5
    offs, tok, expert = plain.route(plain.ids_of(g, T, E, 1, 0.1, dev), E)
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    for dtype in TYPES if a + b <= 6 and K <= 256 else TYPES[::2]:
        y = bgt.w8a8_moe_gemm_fp8(q, s, offs, tok, p["qw"], p["sw"], out_dtype=dtype)
        v = plain.values(q, s)
        for e in range(E):
            i, j = int(offs[e]), int(offs[e + 1])
            if i < j:
                within(y[i:j], v[tok[i:j].long()], plain.matrix(p["qw"][e], p["sw"][e]), dtype)


@pytest.mark.parametrize("dtype", TYPES[::2])
@pytest.mark.parametrize("K", [128, 130])
@pytest.mark.parametrize("g,u,dh", [(-24, 2.0 ** 60, 2.0 ** 80), (-60, 2.0 ** 30, 2.0 ** 120), (-80, 2.0 ** 100, 2.0 ** 120),
                                    (-80, 2.0 ** 120, 2.0 ** 100), (-60, 2.0 ** -80, 2.0 ** 126), (-60, 2.0 ** 126, 2.0 ** -80)])
def test_gate_gradient_in_range(bgt, dev, dtype, K, g, u, dh):
    """Gradients that are finite though dh u or dh g is not, and not lost where one factor is small."""
    rnd = torch.Generator(device=dev).manual_seed(K)
    up = u * (1 + torch.rand(5, K, generator=rnd, device=dev))
    gate = torch.full_like(up, g)
    d = (dh * (1 + torch.rand(5, K, generator=rnd, device=dev))).to(dtype)
    kept = (*bgt.quantize_fp8(gate), *bgt.quantize_fp8(up))
    got = bgt.silu_mul_fp8_backward(d, *kept)
    gv, uv, dd = plain.values(*kept[:2])[:, :K], plain.values(*kept[2:])[:, :K], d.double()
    s = torch.sigmoid(gv)
    for y, ref in zip(got, (dd * uv * s * (1 + gv * (1 - s)), dd * gv * s)):
        assert bool((ref.abs() < torch.finfo(dtype).max).all())
        # at most 32 roundings to fp32: the sigmoid's dozen, the factors and their products. dh of 2^-80
        # times silu(-60) of about 2^-81 lies below the normal range, where a result may be 0.
        assert bool(((y.double() - ref).abs() <= (32 * 2.0 ** -24 + torch.finfo(dtype).eps / 2) * ref.abs() + torch.finfo(dtype).tiny).all())


@pytest.mark.parametrize("dtype", TYPES[::2])
def test_weight_gradient_of_2_32_elements(bgt, dev, dtype):
    """As many outputs as a grid's threads, where no parts are joined: a wide vocabulary's gradient."""
    M, K, N = 4, 1 << 16, 1 << 16
    g = torch.Generator(device=dev).manual_seed(1)
    q, s = bgt.quantize_fp8(torch.randn(M, K, generator=g, device=dev))
    dy = torch.randn(M, N, generator=g, device=dev).to(dtype)
    dw = bgt.wgrad_fp8(q, s, dy)
    assert dw.shape == (K, N)
    x = plain.values(q, s)
    for k in (0, 1, 127, 12345, 32768, 65407, 65535):
        ref, size = x[:, k] @ dy.double(), x[:, k].abs() @ dy.double().abs()
        assert bool(((dw[k].double() - ref).abs() <= M * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * ref.abs()).all())


def whole_numbers(bgt, dev, M, K, N, dtype):
    """Small whole numbers, whose products and sums every instruction holds: outputs are equal to the
    sums rounded once, call after call. A row or group read too early or too late would show."""
    g = torch.Generator(device=dev).manual_seed(M)
    x = torch.randint(-3, 4, (M, K), generator=g, device=dev).float()
    w = torch.randint(-3, 4, (K, N), generator=g, device=dev).float()
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    ref = (x.double() @ w.double()).to(dtype)
    for _ in range(10):
        x.zero_()                                               # other work in between
        y = bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=dtype)
        assert torch.equal(y, ref)


# tiles of 64, 128 and 256; one group of K, an odd and an even number
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(150, 128, 500), (150, 1024, 500), (1030, 640, 3333), (1030, 768, 3333), (2048, 1024, 8200),
                                   (2048, 384, 8200)])
def test_whole_numbers_in_tiles(bgt, dev, dtype, M, K, N):
    whole_numbers(bgt, dev, M, K, N, dtype)


# the streaming kernel: blocks of 16, 32 and 64 rows, fewer and more groups of K than the waves keep
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 128, 300), (5, 512, 300), (9, 4096, 300), (16, 2048, 5000), (30, 2048, 300), (32, 4096, 5000),
                                   (64, 4096, 300), (61, 384, 9000), (16, 8192, 300), (30, 4224, 300), (61, 4608, 300)])
def test_whole_numbers_in_few_rows(bgt, dev, M, K, N, dtype):
    whole_numbers(bgt, dev, M, K, N, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 512, 300), (5, 4096, 300), (8, 2048, 5000)])
def test_whole_numbers_quantized_by_the_product(bgt, dev, M, K, N, dtype):
    g = torch.Generator(device=dev).manual_seed(M)
    w = torch.randint(-3, 4, (K, N), generator=g, device=dev).float()
    p = bgt.pack_weights_fp8(w)
    for _ in range(10):
        x = torch.randint(-3, 4, (M, K), generator=g, device=dev).float()
        y, q, s = bgt.w8a8_linear_fp8(x, p["qw"], p["sw"], out_dtype=dtype)
        assert torch.equal(y, (x.double() @ w.double()).to(dtype)) and torch.equal(plain.values(q, s)[:, :K], x.double())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(64, 256, 256), (1000, 200, 130), (3000, 512, 2048), (600, 2048, 8192)])
def test_whole_numbers_in_weight_gradients(bgt, dev, M, K, N, dtype):
    g = torch.Generator(device=dev).manual_seed(M)
    q, s = bgt.quantize_fp8(torch.randint(-3, 4, (M, K), generator=g, device=dev).float())
    dy = torch.randint(-3, 4, (M, N), generator=g, device=dev).to(dtype)
    ref = (plain.values(q, s)[:, :K].t() @ dy.double()).to(dtype)
    for _ in range(5):
        assert torch.equal(bgt.wgrad_fp8(q, s, dy, K), ref)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 256, 48), (1, 1024, 64), (8, 1024, 64), (30, 1024, 64), (60, 1024, 64), (1, 4224, 48), (20, 4224, 48),
                                   (60, 4224, 48), (300, 1024, 200), (1100, 256, 8200)])
def test_sums_that_cancel(bgt, dev, dtype, M, K, N):
    """Products of 2^16 that cancel, and small ones that are left. Whole numbers, whose sums over 128 (at
    most 2^21) and over K fp32 holds: exact products give the sums rounded once. They are fp32 outputs'
    and those of up to 32 rows of up to 4096. The others lose of each product what lies 13 bits below
    the largest of its group: at most 2^-9 of the magnitudes, and no better is promised."""
    g = torch.Generator(device=dev).manual_seed(M + K)
    x = torch.randint(-3, 4, (M, K), generator=g, device=dev).float()
    w = torch.randint(-3, 4, (K, N), generator=g, device=dev).float()
    x[:, 0::8], x[:, 1::8] = 256.0, -256.0
    w[0::8] = w[1::8] = 256.0
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    xv, wv = plain.values(q, s), plain.matrix(p["qw"], p["sw"])
    assert torch.equal(xv[:, :K], x.double()) and torch.equal(wv[:K], w.double())
    y, ref = bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=dtype), xv @ wv
    if dtype == torch.float32 or (M <= 32 and K <= 4096):
        assert torch.equal(y, ref.to(dtype))
    else:
        bound = plain.product_bound(xv, wv, ref, dtype)
        assert bool(((y.double() - ref).abs() <= bound).all()), float(((y.double() - ref).abs() / bound).max())


# nothing, less than a piece of 16 bytes, whole ones and odd ends; at any alignment of the elements
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N", [(3, 1), (3, 7), (9, 333), (300, 5), (300, 1001)])
def test_rows_behind_the_last_slot(bgt, dev, dtype, T, N):
    """Zeros in the rows without a slot, and nothing written before or behind them."""
    E, K = 4, 128
    g = torch.Generator(device=dev).manual_seed(N)
    q, s = bgt.quantize_fp8(torch.randn(T, K, generator=g, device=dev))
    p = bgt.pack_weights_fp8(torch.randn(E, K, N, generator=g, device=dev))
    for drop in (0.0, 0.3, 1.0):
        offs, tok, expert = plain.route(plain.ids_of(g, T, E, 2, drop, dev), E)
        want = None
        for at in (8, 9, 11, 16):
            room = torch.full((2 * T * N + 40,), 7.0, device=dev, dtype=dtype)
            y = room[at:at + 2 * T * N].view(2 * T, N)
            bgt.w8a8_moe_gemm_fp8(q, s, offs, tok, p["qw"], p["sw"], y=y)
            assert not bool(y[len(expert):].ne(0).any())
            assert bool((room[:at] == 7).all()) and bool((room[at + 2 * T * N:] == 7).all())
            want = y.clone() if want is None else want
            assert torch.equal(y, want)
