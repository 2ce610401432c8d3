"""Products in 8-bit floating point, dense and for routed slots, against 64 bits.

Elementwise within product_bound (what the 8-bit matrix instructions may lose), and over the
whole output within 2^-14 of its norm besides the rounding: products lose bits only where
they are 2^-5 of their group's largest, about 2^-16 of the sum for normal data.
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


def inputs(seed, M, K, N, dev, E=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=dev) * torch.exp2(torch.randint(-3, 4, (M, 1), generator=g, device=dev).float())
    x[:, ::61] *= 20
    w = 0.05 * torch.randn(*([E] if E else []), K, N, generator=g, device=dev)
    return x, w


def check(y, x, w, dtype):
    """y against x.w (doubles)."""
    ref = x @ w
    assert y.dtype == dtype and y.shape == ref.shape
    bound = plain.product_bound(x, w, ref, dtype)
    assert bool(((y.double() - ref).abs() <= bound).all()), float(((y.double() - ref).abs() / bound).max())
    assert plain.rel(y, ref) <= torch.finfo(dtype).eps / 2 + (2.0 ** -20 if dtype == torch.float32 else 2.0 ** -14)


SHAPES = [(1, 128, 16), (1, 4096, 4096), (2, 384, 1), (7, 1000, 333), (16, 256, 130), (17, 2048, 64), (33, 512, 257),
          (61, 4096, 512), (64, 128, 128), (65, 640, 144), (200, 1024, 200), (256, 384, 264), (257, 256, 256),
          (300, 1152, 1000), (513, 130, 129), (1024, 512, 2048), (1500, 4096, 640), (2100, 256, 77)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_dense(bgt, dev, dtype, M, K, N):
    print("dense", M, K, N, dtype, flush=True)
    x, w = inputs(M + K + N, M, K, N, dev)
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w, turned=True)
    check(bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=dtype), plain.values(q, s), plain.matrix(p["qw"], p["sw"]), dtype)
    # the gradient of x: dy.w^T through the turned weights, the same values
    dy = inputs(M, M, N, 1, dev)[0]
    dq, ds = bgt.quantize_fp8(dy)
    turned = plain.matrix(p["qt"], p["st"])
    assert torch.equal(turned[:N], plain.matrix(p["qw"], p["sw"])[:K].t())
    check(bgt.w8a8_gemm_fp8(dq, ds, p["qt"], p["st"], out_dtype=dtype), plain.values(dq, ds), turned, dtype)


@pytest.mark.parametrize("xtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (1, 100, 48), (3, 272, 130), (4, 256, 100), (5, 512, 64), (16, 1024, 256),
                                   (40, 384, 64), (300, 256, 256)])
def test_linear(bgt, dev, xtype, M, K, N):
    """The same codes, scales and outputs as the two calls, for few rows in one launch."""
    x, w = inputs(M * K + N, M, K, N, dev)
    p = bgt.pack_weights_fp8(w)
    x = x.to(xtype)
    for part in (x, torch.cat([x, x], 1)[:, :K], torch.cat([x[:, :1], x], 1)[:, 1:]):   # dense, strided, misaligned
        for dtype in TYPES:
            y, q, s = bgt.w8a8_linear_fp8(part, p["qw"], p["sw"], out_dtype=dtype)
            q2, s2 = bgt.quantize_fp8(part)
            assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
            assert torch.equal(s.view(torch.uint8), s2.view(torch.uint8))
            check(y, plain.values(q, s), plain.matrix(p["qw"], p["sw"]), dtype)
    assert bgt.w8a8_linear_fp8(x, p["qw"], p["sw"])[0].dtype == xtype


# few rows: more blocks of 16 weight rows than workgroups, K longer than the waves keep, each
# count of row blocks; many rows: every tile with one, two and three groups of K and ragged ends
WIDE = [(1, 4096, 9000), (9, 4096, 4400), (17, 4096, 4400), (48, 2048, 6000), (64, 4096, 4400), (1, 5120, 48), (8, 14336, 40),
        (16, 8192, 64), (33, 4224, 40), (61, 14336, 100), (1024, 128, 14336), (1100, 256, 12300), (1030, 300, 12345),
        (1000, 128, 3500), (1000, 200, 3500), (999, 384, 3501), (130, 5000, 1000), (66, 128, 70), (4000, 640, 3333)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", WIDE)
def test_wide(bgt, dev, dtype, M, K, N):
    print("wide", M, K, N, dtype, flush=True)
    x, w = inputs(M + K + N, M, K, N, dev)
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    y = torch.full((M, N), float("nan"), device=dev, dtype=dtype)
    check(bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], y=y), plain.values(q, s), plain.matrix(p["qw"], p["sw"]), dtype)


ROUTED = [(1, 8, 2, 0.0, 512, 256), (3, 4, 1, 0.0, 128, 100), (16, 8, 2, 0.0, 1024, 512), (61, 5, 3, 0.2, 384, 129),
          (100, 3, 2, 0.5, 130, 64), (300, 4, 2, 0.1, 256, 272), (1000, 2, 1, 0.0, 512, 300), (700, 64, 4, 0.1, 256, 96),
          (9, 4, 2, 1.0, 256, 64), (20, 4, 2, 0.0, 5000, 200), (40, 8, 2, 0.1, 1024, 4400), (1500, 2, 1, 0.1, 128, 10000),
          (1600, 2, 1, 0.0, 384, 10001), (400, 4, 2, 0.1, 256, 3400), (3, 4, 2, 0.0, 8192, 48)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,drop,K,N", ROUTED)
def test_routed(bgt, dev, dtype, T, E, k, drop, K, N):
    print("routed", T, E, k, K, N, dtype, flush=True)
    x, w = inputs(T + E + K + N, T, K, N, dev, E)
    g = torch.Generator(device=dev).manual_seed(T)
    offs, tok, expert = plain.route(plain.ids_of(g, T, E, k, drop, dev), E)
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w)
    y = torch.full((T * k, N), float("nan"), device=dev, dtype=dtype)
    bgt.w8a8_moe_gemm_fp8(q, s, offs, tok, p["qw"], p["sw"], y=y)
    n, v = len(expert), plain.values(q, s)
    assert not bool(y[n:].ne(0).any())                        # slots past the last expert's
    for e in range(E):
        a, b = int(offs[e]), int(offs[e + 1])
        if a < b:
            check(y[a:b], v[tok[a:b].long()], plain.matrix(p["qw"][e], p["sw"][e]), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_not_finite_blocks(bgt, dev, dtype, M):
    """A row's block that is not finite makes that row NaN and no other; of a weight's block its
    128 outputs."""
    x, w = inputs(M, M, 512, 300, dev)
    clean = bgt.w8a8_gemm_fp8(*bgt.quantize_fp8(x), *bgt.pack_weights_fp8(w).values(), out_dtype=dtype)
    x[M // 2, 200] = float("inf")
    y = bgt.w8a8_gemm_fp8(*bgt.quantize_fp8(x), *bgt.pack_weights_fp8(w).values(), out_dtype=dtype)
    assert bool(y[M // 2].isnan().all())
    y[M // 2] = clean[M // 2]
    assert torch.equal(y, clean)
    x[M // 2, 200] = 0
    w[300, 130] = float("nan")
    y = bgt.w8a8_gemm_fp8(*bgt.quantize_fp8(x), *bgt.pack_weights_fp8(w).values(), out_dtype=dtype)
    assert bool(y[:, 128:256].isnan().all()) and not bool(y[:, :128].isnan().any()) and not bool(y[:, 256:].isnan().any())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_large_and_small_scales(bgt, dev, M):
    """Blocks of very different powers of two: the fp32 sums hold them, also where one factor is
    far outside the type."""
    g = torch.Generator(device=dev).manual_seed(M)
    K, N = 256, 48
    x = torch.randn(M, K, generator=g, device=dev) * 2.0 ** 60
    w = torch.randn(K, N, generator=g, device=dev) * 2.0 ** -60
    x[:, 128:] *= 2.0 ** -90
    w[128:] *= 2.0 ** 90
    q, s = bgt.quantize_fp8(x)
    w2 = bgt.pack_weights_fp8(w)
    for dtype in TYPES:
        check(bgt.w8a8_gemm_fp8(q, s, w2["qw"], w2["sw"], out_dtype=dtype), plain.values(q, s), plain.matrix(w2["qw"], w2["sw"]), dtype)


def test_equal_bits_and_streams(bgt, dev):
    """Equal inputs give equal bits, on two streams at once too."""
    cases = []
    for M, K, N in ((1, 4096, 512), (61, 1024, 256), (700, 1024, 512)):
        x, w = inputs(M, M, K, N, dev)
        q, s = bgt.quantize_fp8(x)
        cases.append((q, s, *bgt.pack_weights_fp8(w).values()))
    ref = [bgt.w8a8_gemm_fp8(*c, out_dtype=torch.bfloat16) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append([bgt.w8a8_gemm_fp8(*c, out_dtype=torch.bfloat16) for c in cases])
        torch.cuda.synchronize()
        for out in got:
            for a, b in zip(out, ref):
                assert torch.equal(a, b)


def test_many_elements(bgt, dev):
    """Codes past 2^31 bytes, rows of y past 2^31 elements."""
    M, K, N = (1 << 18) + 70, 8192, 8200
    q = torch.zeros(M, K, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.full((K // 128, M), 127, device=dev, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    x, w = inputs(3, 80, K, N, dev)
    a, b = bgt.quantize_fp8(x)
    q[-80:].view(torch.uint8).copy_(a.view(torch.uint8))
    s.view(torch.uint8)[:, -80:].copy_(b.view(torch.uint8))
    p = bgt.pack_weights_fp8(w)
    y = bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=torch.bfloat16)
    check(y[-80:], plain.values(a, b), plain.matrix(p["qw"], p["sw"]), torch.bfloat16)
    assert not bool(y[:1000].any()) and not bool(y[-180:-80].any())


@pytest.mark.parametrize("more", [18, 19])
def test_many_routed_elements(bgt, dev, more):
    """Codes of routed rows past 2^31 and past 2^32 bytes."""
    T, K, N = (1 << more) + 70, 8192, 256
    q = torch.zeros(T, K, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.full((K // 128, T), 127, device=dev, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    x, w = inputs(more, 80, K, N, dev, 2)
    a, b = bgt.quantize_fp8(x)
    q[-80:].view(torch.uint8).copy_(a.view(torch.uint8))
    s.view(torch.uint8)[:, -80:].copy_(b.view(torch.uint8))
    p = bgt.pack_weights_fp8(w)
    offs = torch.tensor([0, T // 2, T], dtype=torch.int32, device=dev)
    tok = torch.arange(T, dtype=torch.int32, device=dev)
    y = bgt.w8a8_moe_gemm_fp8(q, s, offs, tok, p["qw"], p["sw"], out_dtype=torch.bfloat16)
    check(y[-80:], plain.values(a, b), plain.matrix(p["qw"][1], p["sw"][1]), torch.bfloat16)
    assert not bool(y[:-80].any())


def test_refusals(bgt, dev):
    """What the Python functions refuse: shapes that do not fit each other, other dtypes."""
    x, w = inputs(1, 8, 256, 64, dev)
    q, s = bgt.quantize_fp8(x)
    p = bgt.pack_weights_fp8(w, turned=True)
    offs = torch.tensor([0, 4, 8], dtype=torch.int32, device=dev)
    tok = torch.arange(8, dtype=torch.int32, device=dev)
    for call in (lambda: bgt.w8a8_gemm_fp8(q[:, :128].contiguous(), s, p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s[:, :4].contiguous(), p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s, p["qt"], p["st"]), lambda: bgt.w8a8_gemm_fp8(q, s, p["qw"], p["st"]),
                 lambda: bgt.w8a8_gemm_fp8(q[::2], s, p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], y=torch.empty(8, 65, device=dev)),
                 lambda: bgt.w8a8_linear_fp8(x[:, :100], p["qw"], p["sw"]),
                 lambda: bgt.w8a8_moe_gemm_fp8(q, s, offs, tok, p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s.cpu(), p["qw"], p["sw"]),
                 lambda: bgt.wgrad_fp8(q, s, x[:4]), lambda: bgt.wgrad_fp8(q, s, x, K=100),
                 lambda: bgt.moe_wgrad_fp8(q, s, offs, tok, x[:4]),
                 lambda: bgt.silu_mul_fp8(x, x[:, :128]), lambda: bgt.silu_mul_fp8(x, x.half()),
                 lambda: bgt.silu_mul_fp8_backward(x[:4], q, s, q, s),
                 lambda: bgt.dequantize_fp8(q, s, 100), lambda: bgt.pack_weights_fp8(w.t()),
                 lambda: bgt.pack_weights_fp8(w, qt=p["qt"])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bgt.quantize_fp8(x.double()), lambda: bgt.quantize_fp8(tok.view(2, 4)),
                 lambda: bgt.w8a8_gemm_fp8(q.view(torch.uint8), s, p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s.view(torch.uint8), p["qw"], p["sw"]),
                 lambda: bgt.w8a8_gemm_fp8(q, s, p["qw"], p["sw"], out_dtype=torch.float64),
                 lambda: bgt.moe_balance(x.double(), tok.view(8, 1)), lambda: bgt.moe_balance(x, tok.view(8, 1).long())):
        with pytest.raises(TypeError):
            call()


def test_graph(bgt, dev):
    """Captured and replayed with eager work between the replays: every operator that makes up a
    layer's step, workspaces among them."""
    x, w = inputs(1, 300, 384, 256, dev)
    dy, logits = inputs(2, 300, 256, 1, dev)[0].to(torch.bfloat16), inputs(3, 300, 8, 1, dev)[0]
    x = x.to(torch.bfloat16)
    ids = torch.randint(0, 8, (300, 2), dtype=torch.int32, device=dev)
    long_x = inputs(4, 2100, 256, 1, dev)[0].to(torch.bfloat16)
    one = torch.ones((), device=dev)

    def step():
        p = bgt.pack_weights_fp8(w, turned=True)
        y, q, s = bgt.w8a8_linear_fp8(x, p["qw"], p["sw"])
        y1 = bgt.w8a8_linear_fp8(x[:1], p["qw"], p["sw"])[0]
        kept = bgt.silu_mul_fp8(y, y)
        dg, du = bgt.silu_mul_fp8_backward(dy, *kept[2:])
        dx = bgt.w8a8_linear_fp8(dg, p["qt"], p["st"])[0]
        lq, ls = bgt.quantize_fp8(long_x)
        out = bgt.moe_balance(logits, ids)
        return (y, y1, *kept, dg, du, dx, bgt.wgrad_fp8(q, s, dy), bgt.wgrad_fp8(lq, ls, long_x), bgt.dequantize_fp8(q, s),
                *out, bgt.moe_balance_backward(one, logits, out[1], out[3]))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.mul_(1.5)
        w.mul_(0.5)
        logits.add_(torch.randn_like(logits))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a, b.view(torch.uint8) if b.element_size() == 1 else b)
