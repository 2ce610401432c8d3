"""Few rows of unquantized activations times 4-bit weights, against 64 bits.

y_ij = sum_l s_lj sum_{k in group l} x_ik q_kj for fp32, fp16 and bf16 x and
every output type, dense and for routed slots: one row to more than one pass,
one group to 112, ragged column counts, strides and unaligned rows, codes of -8,
zero scales, infinities and NaN, malformed routing, sizes past 2^32 bytes.

Bound: x and q are exact in every product, so an output differs from the exact
value by the fp32 additions: at most 128 in a group, G across the groups and 64
joins, each at most one ulp of the running sum's bound (matrix cores may
truncate), plus the output's rounding.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}


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


def say(*a):
    print(*a, flush=True)


def weights(bgt, dev, seed, K, N):
    """Random codes -8..7, their packed form, scales (some groups zero), and W in 64 bits."""
    g = torch.Generator(device=dev).manual_seed(seed)
    q = torch.randint(-8, 8, (K, N), generator=g, device=dev)
    canonical = (q.t() & 15).reshape(N, K // 2, 2)
    canonical = (canonical[..., 0] | canonical[..., 1] << 4).to(torch.uint8).reshape(-1).contiguous()
    packed = bgt.repack_int4_canonical(canonical, K, N)
    s = 0.01 * torch.rand(K // 128, N, generator=g, device=dev)
    s[torch.rand(K // 128, N, generator=g, device=dev) < 0.05] = 0.0
    return packed, s, q.double() * s.double().repeat_interleave(128, 0)


def rows_of(seed, M, K, dt, dev):
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x = torch.randn(M, K, generator=g, device=dev)
    x[:, torch.randperm(K, generator=g, device=dev)[: max(1, K // 100)]] *= 20
    return x.to(dt)


def check(y, x, W):
    xd = x.double()
    ref = xd @ W
    size = xd.abs() @ W.abs()
    G = W.shape[0] // 128
    tol = 2 * (128 + G + 64) * U * size + ref.abs() * HALF_ULP[y.dtype] + TINY[y.dtype]
    bad = (y.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off"


DENSE = [(1, 128, 16), (1, 4096, 4096), (2, 256, 48), (3, 11008, 208), (5, 4096, 64), (6, 512, 80),
         (15, 640, 144), (16, 4096, 4112), (17, 1152, 96), (21, 384, 32), (22, 896, 160),
         (32, 2048, 1024), (33, 4096, 48), (48, 768, 272), (64, 14336, 64), (65, 512, 112),
         (130, 1024, 400), (4, 14336, 4096), (1, 65536, 16), (1, 2048, 22016), (31, 11008, 1376)]


@pytest.mark.parametrize("M,K,N", DENSE)
@pytest.mark.parametrize("kind", list(TYPES))
def test_dense(bgt, dev, M, K, N, kind):
    say(f"gemv M={M} K={K} N={N} {kind}")
    packed, s, W = weights(bgt, dev, M + K + N, K, N)
    x = rows_of(M * K, M, K, TYPES[kind], dev)
    y = bgt.w4a16_gemv(x, packed, s, N)
    assert y.dtype == x.dtype and y.shape == (M, N)
    check(y, x, W)


@pytest.mark.parametrize("M", [1, 5, 9, 30, 40])
@pytest.mark.parametrize("tiles", [255, 257, 601, 901, 1100])
@pytest.mark.parametrize("kind", list(TYPES))
def test_many_tiles(bgt, dev, M, tiles, kind):
    # one to four column tiles a workgroup, the last one partly past the end, and
    # group counts that the waves share unevenly
    K, N = (384, 640, 128)[tiles % 3], 16 * tiles
    say(f"gemv M={M} K={K} N={N} {kind}")
    packed, s, W = weights(bgt, dev, M + tiles, K, N)
    x = rows_of(M * K, M, K, TYPES[kind], dev)
    check(bgt.w4a16_gemv(x, packed, s, N), x, W)


@pytest.mark.parametrize("rows", [1, 4, 5, 16, 17, 24, 25, 32, 33, 70])
@pytest.mark.parametrize("kind", list(TYPES))
def test_routed_row_counts(bgt, dev, rows, kind):
    # one expert with `rows` slots beside experts with fewer: every row block size
    # and several passes
    say(f"moe gemv one expert with {rows} rows {kind}")
    ids = np.full((rows, 1), 2, np.int32)
    check_moe(bgt, dev, ids, 3, 256, 16 * 301, TYPES[kind], rows)
    wide = np.stack([np.full(rows, 1), np.arange(rows) % 4 + 2], 1).astype(np.int32)
    check_moe(bgt, dev, wide, 6, 640, 48, TYPES[kind], rows + 1)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
def test_output_types_and_packer(bgt, dev, kind, out):
    # the packer's own codes and scales
    M, K, N = 7, 1024, 304
    w = 0.02 * torch.randn(K, N, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    pw = bgt.pack_weights_int4(w)
    v = (w.view(K // 128, 128, N) / pw["fscale"][:, None]).view(K, N).double()
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)           # half away from zero, as the packer
    W = q.double() * pw["fscale"].double().repeat_interleave(128, 0)
    x = rows_of(3, M, K, TYPES[kind], dev)
    y = bgt.w4a16_gemv(x, pw["packed"], pw["fscale"], N, out_dtype=TYPES[out])
    assert y.dtype == TYPES[out]
    check(y, x, W)


@pytest.mark.parametrize("kind", list(TYPES))
def test_strides_and_unaligned_rows(bgt, dev, kind):
    K, N = 512, 96
    packed, s, W = weights(bgt, dev, 5, K, N)
    full = rows_of(5, 40, 600, TYPES[kind], dev)
    for x in (full[:20, :K], full[::2, 8:8 + K], full[:9, 1:1 + K], full[3:4, 7:7 + K], full[:18, 3:3 + K]):
        check(bgt.w4a16_gemv(x, packed, s, N), x, W)


@pytest.mark.parametrize("kind", list(TYPES))
def test_small_and_large_values(bgt, dev, kind):
    # subnormal and near-largest elements
    dt = TYPES[kind]
    K, N = 256, 64
    packed, s, W = weights(bgt, dev, 8, K, N)
    fi = torch.finfo(dt)
    x = rows_of(8, 6, K, dt, dev)
    x[0] = fi.max * (0.5 if kind == "f16" else 2.0 ** -12)
    x[1] = (fi.tiny * 8 * torch.rand(K, device=dev)).to(dt)
    x[2] = 0
    y = bgt.w4a16_gemv(x, packed, s, N, out_dtype=torch.float32)
    xd = x.double()
    ref, size = xd @ W, xd.abs() @ W.abs()
    tol = 2 * (128 + 2 + 64) * U * size
    if kind == "f16":
        assert ((y.double() - ref).abs() <= tol + 1e-37)[1].all()      # fp16 subnormals count
    # fp32 and bf16 subnormals (below 2^-126) may be taken as zero
    keep = [0, 2, 3, 4, 5]
    assert ((y.double() - ref).abs() <= tol + 1e-37)[keep].all()
    assert ((y.double() - ref).abs()[1] <= tol[1] + K * 8 * 0.01 * 2.0 ** -126).all()
    assert (y[2] == 0).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_infinities_and_nan_stay_in_their_rows(bgt, dev, kind):
    M, K, N = 19, 512, 48
    packed, s, W = weights(bgt, dev, 9, K, N)
    x = rows_of(9, M, K, TYPES[kind], dev)
    x[4, 100] = float("inf")
    x[11, 300] = float("nan")
    x[18, 7] = float("-inf")
    y = bgt.w4a16_gemv(x, packed, s, N).double()
    fine = [i for i in range(M) if i not in (4, 11, 18)]
    ok = x[fine]
    check(bgt.w4a16_gemv(ok.contiguous(), packed, s, N), ok, W)
    assert torch.isfinite(y[fine]).all()
    assert torch.equal(y[fine], bgt.w4a16_gemv(x.nan_to_num(0, 0, 0), packed, s, N).double()[fine])
    assert torch.isnan(y[11]).all()
    if kind == "f32":                              # a signaling NaN, its payload in the low bits only
        x[11, 300] = torch.tensor(0x7F800001, dtype=torch.int32).view(torch.float32)
        assert torch.isnan(bgt.w4a16_gemv(x, packed, s, N)[11]).all()
    for row, k, sign in ((4, 100, 1), (18, 7, -1)):
        w = W[k]                                   # inf times a code: its sign, or NaN for 0
        assert torch.equal(torch.isnan(y[row]), w == 0)
        assert torch.equal(y[row][w != 0], sign * torch.sign(w[w != 0]) * float("inf"))


def slots(T, E, k, seed, drop=0.0, only=None):
    g = np.random.default_rng(seed)
    ids = np.argsort(g.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if only is not None:
        ids = np.full((T, 1), only, np.int32)
    ids[g.random(ids.shape) < drop] = -1
    return ids


def check_moe(bgt, dev, ids, E, K, N, dt, seed, out=None):
    offs, tok, _ = bgt.moe_sort(torch.from_numpy(ids).to(dev), E)
    T = ids.shape[0]
    x = rows_of(seed, T, K, dt, dev)
    made = [weights(bgt, dev, seed + 10 * e, K, N) for e in range(E)]
    packed = torch.stack([m[0] for m in made])
    s = torch.stack([m[1] for m in made])
    y = torch.full((tok.numel(), N), float("nan"), dtype=out or dt, device=dev)
    bgt.w4a16_moe_gemv(x, offs, tok, packed, s, N, y=y)
    o = offs.tolist()
    for e in range(E):
        if o[e] < o[e + 1]:
            check(y[o[e]:o[e + 1]], x[tok[o[e]:o[e + 1]].long()], made[e][2])
    assert (y[o[E]:] == 0).all()


@pytest.mark.parametrize("T,E,k,K,N", [(1, 8, 2, 4096, 64), (2, 4, 1, 128, 16), (5, 8, 2, 1024, 208),
                                       (16, 8, 2, 2048, 96), (61, 8, 2, 1152, 48), (64, 4, 4, 512, 112),
                                       (9, 64, 8, 256, 32), (130, 3, 2, 384, 80), (33, 2, 2, 14336, 16),
                                       (7, 200, 3, 128, 64)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_routed(bgt, dev, T, E, k, K, N, kind):
    say(f"moe gemv T={T} E={E} k={k} K={K} N={N} {kind}")
    check_moe(bgt, dev, slots(T, E, k, T + E), E, K, N, TYPES[kind], T + K)


@pytest.mark.parametrize("kind", list(TYPES))
def test_routed_dropped_and_skewed(bgt, dev, kind):
    dt = TYPES[kind]
    check_moe(bgt, dev, slots(30, 8, 2, 1, drop=0.4), 8, 256, 80, dt, 1)
    check_moe(bgt, dev, slots(70, 8, 1, 2, only=5), 8, 256, 48, dt, 2)
    check_moe(bgt, dev, slots(6, 4, 2, 3, drop=1.0), 4, 128, 32, dt, 3)
    check_moe(bgt, dev, slots(12, 8, 2, 4), 8, 640, 144, dt, 4, out=torch.float32)


@pytest.mark.parametrize("counts", [[33, 1, 16, 17, 0, 24, 25, 6], [61, 9, 9, 9, 9, 9, 8, 8], [32] * 4,
                                    [0, 65, 0, 64, 1], [200, 0, 1, 130], [0] * 70 + [40] + [1] * 30 + [90, 0, 35]])
@pytest.mark.parametrize("kind", list(TYPES))
def test_experts_of_several_passes(bgt, dev, counts, kind):
    """Experts with more slots than one pass takes, next to ones with few or none."""
    say(f"moe gemv counts={counts} {kind}")
    ids = np.repeat(np.arange(len(counts), dtype=np.int32), counts)[:, None]
    np.random.default_rng(len(ids)).shuffle(ids)
    check_moe(bgt, dev, ids, len(counts), 256, 48, TYPES[kind], len(ids))


def test_routing_that_points_outside(bgt, dev):
    # offsets and tokens are clamped: nothing outside the buffers is touched
    T, E, K, N, R = 4, 3, 256, 32, 8
    made = [weights(bgt, dev, e, K, N) for e in range(E)]
    packed, s = torch.stack([m[0] for m in made]), torch.stack([m[1] for m in made])
    x = rows_of(1, T, K, torch.bfloat16, dev)
    offs = torch.tensor([-5, 2, 1000, 3], dtype=torch.int32, device=dev)
    tok = torch.tensor([-9, 1, 10 ** 9, 2, 0, 3, 1, 2], dtype=torch.int32, device=dev)
    y = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    bgt.w4a16_moe_gemv(x, offs, tok, packed, s, N, y=y)
    torch.cuda.synchronize()
    check(y[:2], x[[0, 1]], made[0][2])


def test_weights_past_32_bits(bgt, dev):
    # 48 experts of 98 MiB: the last one starts past 2^32 bytes
    E, K, N, T = 48, 14336, 14336, 2
    packed = torch.empty(E, N * K // 2, dtype=torch.uint8, device=dev)
    s = torch.full((E, K // 128, N), 0.01, device=dev)
    assert (E - 1) * N * K // 2 > 2 ** 32
    packed.zero_()
    one, so, _ = weights(bgt, dev, 1, K, 64)        # 4 column tiles, put at the end of the last expert
    packed[E - 1, -one.numel():] = one
    s[E - 1, :, -64:] = so
    W = weights(bgt, dev, 1, K, 64)[2]
    x = rows_of(2, T, K, torch.bfloat16, dev)
    ids = torch.tensor([[0, E - 1], [E - 1, 3]], dtype=torch.int32, device=dev)
    offs, tok, pos = bgt.moe_sort(ids, E)
    y = bgt.w4a16_moe_gemv(x, offs, tok, packed, s, N)
    lo = int(offs[E - 1])
    check(y[lo:, -64:], x[tok[lo:].long()], W)
    assert (y[lo:, :-64] == 0).all() and (y[:lo] == 0).all()


def test_repeatable_other_stream_and_graph(bgt, dev):
    K, N, T, E, k = 2048, 512, 24, 8, 2
    packed, s, W = weights(bgt, dev, 3, K, N)
    xs = [rows_of(i, T, K, torch.bfloat16, dev) for i in range(3)]
    eager = [bgt.w4a16_gemv(x, packed, s, N) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [bgt.w4a16_gemv(x, packed, s, N) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    # routing, experts and combine in one graph
    pk, fs = torch.stack([packed] * E), torch.stack([s] * E)
    logits = [torch.randn(T, E, device=dev) for _ in range(3)]

    def layer(x, v):
        w, ids, offs, tok, pos = bgt.moe_route(v, k)
        return bgt.moe_combine(bgt.w4a16_moe_gemv(x, offs, tok, pk, fs, N), pos, w)

    eager = [layer(x, v) for x, v in zip(xs, logits)]
    bx, bv = xs[0].clone(), logits[0].clone()
    layer(bx, bv)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(bx, bv)
    for i in (1, 2, 0, 1):
        bx.copy_(xs[i])
        bv.copy_(logits[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])


def test_refusals(bgt, dev):
    packed, s, _ = weights(bgt, dev, 1, 256, 32)
    x = torch.randn(2, 256, device=dev)
    with pytest.raises(bgt.BgtError):
        bgt.w4a16_gemv(torch.empty(0, 256, device=dev), packed, s, 32)
    with pytest.raises(ValueError):
        bgt.w4a16_gemv(x, packed, s, 48)
    with pytest.raises(ValueError):
        bgt.w4a16_gemv(x.t(), packed, s, 32)
    with pytest.raises(TypeError):
        bgt.w4a16_gemv(x.double(), packed, s, 32)
    with pytest.raises(TypeError):
        bgt.w4a16_gemv(x, packed, s.half(), 32)
    with pytest.raises(TypeError):
        bgt.w4a16_gemv(x, packed, s, 32, out_dtype=torch.int32)
    with pytest.raises(bgt.BgtError) as e:
        bgt.w4a16_gemv(x[:1].expand(2, 256), packed, s, 32)
    assert e.value.status == bgt.BGT_ERR_SHAPE
    with pytest.raises(bgt.BgtError):             # K not a multiple of the group
        bgt.w4a16_gemv(torch.randn(2, 192, device=dev), torch.zeros(192 * 16, dtype=torch.uint8, device=dev),
                       torch.zeros(1, 32, device=dev), 32)
    offs = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    tok = torch.zeros(2, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        bgt.w4a16_moe_gemv(x, offs, tok, packed, s, 32)
    with pytest.raises(TypeError):
        bgt.w4a16_moe_gemv(x, offs.long(), tok, torch.stack([packed] * 2), torch.stack([s] * 2), 32)
