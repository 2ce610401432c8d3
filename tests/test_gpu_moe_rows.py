"""Token rows to expert order and back, and the gradients, against 64 bits.

The copy is exact; sums lie within bounds derived from fp32 accumulation and
one rounding of the output. Row lengths cover one element, odd ones (the
element path) and whole 16-byte multiples (the wide path); tokens without
experts, strides, unaligned bases, infinities in dropped rows, and sizes
past 2^31 elements.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}    # rounding of the output
TINY = {"f32": 1e-37, "f16": 2.0 ** -25, "bf16": 1e-37}


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


def routing(bgt, dev, T, E, k, seed, drop=0.2):
    """Sorted slots of random distinct experts; some dropped, one token wholly."""
    g = np.random.default_rng(seed)
    ids = np.argsort(g.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[g.random((T, k)) < drop] = -1
    if drop and T > 1:
        ids[T // 2] = -1
    offs, tok, pos = bgt.moe_sort(torch.from_numpy(ids).to(dev), E)
    return offs, tok, pos


SHAPES = [(1, 1, 1, 1), (1, 4096, 8, 2), (5, 7, 4, 3), (16, 4096, 8, 2), (33, 1000, 60, 4),
          (100, 64, 8, 8), (61, 2048, 16, 1), (257, 65, 8, 2), (40, 8200, 8, 2), (19, 14336, 4, 2),
          (2000, 136, 64, 6), (700, 4104, 8, 2), (12, 513, 32, 16)]


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_gather_and_back(bgt, dev, T, H, E, k, kind):
    say(f"gather T={T} H={H} E={E} k={k} {kind}")
    offs, tok, pos = routing(bgt, dev, T, E, k, T + H)
    g = torch.Generator(device=dev).manual_seed(T * 3 + H)
    x = torch.randn(T, H, generator=g, device=dev).to(TYPES[kind])
    xs = bgt.moe_gather(x, offs, pos, xs=torch.full((T * k, H), 7.0, dtype=x.dtype, device=dev))
    want = torch.where(tok[:, None] >= 0, x[tok.clamp(min=0).long()], torch.zeros_like(x[:1]))
    assert torch.equal(xs, want)
    # the gradient: rows summed back; dropped rows hold infinities nobody may read
    dxs = torch.randn(T * k, H, generator=g, device=dev).to(TYPES[kind])
    dxs[int(offs[-1]):] = float("inf")
    dx = bgt.moe_gather_backward(dxs, pos)
    rows = torch.where(pos[..., None] >= 0, dxs[pos.clamp(min=0).long()].double(), 0.0)
    ref = rows.sum(1)
    tol = k * U * rows.abs().sum(1) + ref.abs() * HALF_ULP[kind] + TINY[kind]
    assert ((dx.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_combine_and_gradients(bgt, dev, T, H, E, k, kind):
    say(f"combine T={T} H={H} E={E} k={k} {kind}")
    offs, tok, pos = routing(bgt, dev, T, E, k, T + 2 * H)
    g = torch.Generator(device=dev).manual_seed(T * 5 + H)
    ys = torch.randn(T * k, H, generator=g, device=dev).to(TYPES[kind])
    ys[int(offs[-1]):] = float("nan")
    w = torch.rand(T, k, generator=g, device=dev)
    w[pos < 0] = 0.0
    y = bgt.moe_combine(ys, pos, w)
    there = pos[..., None] >= 0
    rows = torch.where(there, ys[pos.clamp(min=0).long()].double(), 0.0)
    wd = w.double()[..., None]
    ref = (wd * rows).sum(1)
    tol = (k + 1) * U * (wd * rows.abs()).sum(1) + ref.abs() * HALF_ULP[kind] + TINY[kind]
    assert y.dtype == ys.dtype
    assert ((y.double() - ref).abs() <= tol).all()

    dy = torch.randn(T, H, generator=g, device=dev).to(TYPES[kind])
    dys, dw = bgt.moe_combine_backward(dy, ys, offs, pos, w)
    wr = torch.zeros(T * k, dtype=torch.float64, device=dev)
    wr[pos[pos >= 0].long()] = w[pos >= 0].double()
    want = torch.where(tok[:, None] >= 0, wr[:, None] * dy.double()[tok.clamp(min=0).long()], 0.0)
    assert ((dys.double() - want).abs() <= want.abs() * (HALF_ULP[kind] + U) + TINY[kind]).all()
    prod = rows * dy.double()[:, None]
    # the longest chain of one output: a lane's share of the row and the joins
    tol = (H / 32 + 32) * U * prod.abs().sum(2) + 1e-37
    assert ((dw.double() - prod.sum(2)).abs() <= tol).all()


@pytest.mark.parametrize("T,H,E,k", [(1, 8192, 8, 8), (3, 4104, 16, 7), (2, 100, 32, 16),
                                     (70, 4096, 16, 5), (300, 8192, 8, 3)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_combine_gradient_of_few_tokens(bgt, dev, T, H, E, k, kind):
    """Few tokens (whose places may go to several workgroups) and the same tokens
    among many have gradients of the same bits."""
    say(f"combine's gradient, few tokens T={T} H={H} E={E} k={k} {kind}")
    many = 600
    g = torch.Generator(device=dev).manual_seed(T + H + k)
    ids = torch.rand(many, E, generator=g, device=dev).argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand(many, k, generator=g, device=dev) < 0.1] = -1
    rows = torch.randn(many, k, H, generator=g, device=dev).to(TYPES[kind])
    dy = torch.randn(many, H, generator=g, device=dev).to(TYPES[kind])
    w = torch.rand(many, k, generator=g, device=dev)
    got = []
    for n in (T, many):
        offs, tok, pos = bgt.moe_sort(ids[:n].contiguous(), E)
        ys = torch.full((n * k, H), float("nan"), dtype=TYPES[kind], device=dev)
        there = pos >= 0
        ys[pos[there].long()] = rows[:n][there]
        dys, dw = bgt.moe_combine_backward(dy[:n], ys, offs, pos, w[:n])
        assert (dys[int(offs[-1]):] == 0).all() and (dw[~there] == 0).all()
        got.append((dys[pos[:T].clamp(min=0).long()][there[:T]], dw[:T]))
        prod = (rows[:n].double() * dy[:n].double()[:, None]) * there[..., None]
        tol = (H / 32 + 32) * U * prod.abs().sum(2) + 1e-37
        assert ((dw.double() - prod.sum(2)).abs() <= tol).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_combine_gradient_against_differences(bgt, dev):
    # f(ys, w) = <dy, combine(ys, w)> is linear in each: differences are exact
    # up to rounding
    T, H, E, k = 9, 40, 5, 3
    offs, tok, pos = routing(bgt, dev, T, E, k, 1)
    g = torch.Generator(device=dev).manual_seed(2)
    ys = torch.randn(T * k, H, generator=g, device=dev)
    ys[int(offs[-1]):] = 0
    w = torch.rand(T, k, generator=g, device=dev).masked_fill(pos < 0, 0.0)
    dy = torch.randn(T, H, generator=g, device=dev)
    dys, dw = bgt.moe_combine_backward(dy, ys, offs, pos, w)

    def f(a, b):
        return (bgt.moe_combine(a, pos, b).double() * dy.double()).sum()

    size = (bgt.moe_combine(ys.abs(), pos, w).double() * dy.abs().double()).sum()
    for t, i in ((0, 0), (3, 2), (8, 1), (4, 0)):
        step = torch.zeros_like(w)
        step[t, i] = 0.5
        diff = f(ys, w + step) - f(ys, w - step)
        assert abs(float(diff - dw[t, i])) <= 16 * U * float(size + dw.abs().max() * 4)
    for r, h in ((0, 0), (5, 17), (int(offs[-1]) - 1, 39)):
        step = torch.zeros_like(ys)
        step[r, h] = 0.5
        diff = f(ys + step, w) - f(ys - step, w)
        assert abs(float(diff - dys[r, h])) <= 16 * U * float(size + 4)


def test_strides_and_unaligned_bases(bgt, dev):
    T, E, k = 50, 8, 2
    offs, tok, pos = routing(bgt, dev, T, E, k, 4)
    for kind, dt in TYPES.items():
        full = torch.randn(T, 300, device=dev).to(dt)
        for view in (full[:, :256], full[:, 8:264], full[:, 1:257], full[:, 3:250]):
            H = view.shape[1]
            xs = bgt.moe_gather(view, offs, pos)
            want = torch.where(tok[:, None] >= 0, view[tok.clamp(min=0).long()], torch.zeros(1, dtype=dt, device=dev))
            assert torch.equal(xs, want)
            ys = torch.randn(T * k, H, device=dev).to(dt)
            w = torch.rand(T, k, device=dev)
            a = bgt.moe_combine_backward(view, ys, offs, pos, w)
            b = bgt.moe_combine_backward(view.contiguous(), ys, offs, pos, w)
            assert torch.equal(a[0], b[0])
            assert torch.allclose(a[1], b[1], rtol=0, atol=64 * U * float(a[1].abs().max() + 256))


def test_no_experts_at_all(bgt, dev):
    ids = torch.full((6, 2), -1, dtype=torch.int32, device=dev)
    offs, tok, pos = bgt.moe_sort(ids, 4)
    x = torch.randn(6, 32, device=dev)
    assert (bgt.moe_gather(x, offs, pos) == 0).all()
    nan = torch.full((12, 32), float("nan"), device=dev)
    w = torch.zeros(6, 2, device=dev)
    assert (bgt.moe_combine(nan, pos, w) == 0).all()
    dys, dw = bgt.moe_combine_backward(x, nan, offs, pos, w)
    assert (dys == 0).all() and (dw == 0).all()


def test_lists_that_point_outside(bgt, dev):
    # positions outside the slots are skipped, an offset past them is clamped
    T, H = 8, 64
    x = torch.randn(T, H, device=dev)
    pos = torch.tensor([[t, 1000 + t] for t in range(T)], dtype=torch.int32, device=dev)
    offs = torch.tensor([0, 0, 10 ** 6], dtype=torch.int32, device=dev)
    xs = bgt.moe_gather(x, offs, pos, xs=torch.full((2 * T, H), 3.0, device=dev))
    assert torch.equal(xs[:T], x) and (xs[T:] == 3.0).all()
    assert torch.equal(bgt.moe_gather_backward(xs, pos), x)


def test_offsets_past_32_bits(bgt, dev):
    # more than 2^31 elements (2^32 bytes) of rows; sampled rows
    T, H, E, k = 262200, 4104, 8, 2
    g = torch.Generator(device=dev).manual_seed(9)
    ids = torch.stack([torch.randint(0, 4, (T,), generator=g, device=dev),
                       torch.randint(4, 8, (T,), generator=g, device=dev)], 1).to(torch.int32)
    offs, tok, pos = bgt.moe_sort(ids, E)
    assert T * k * H > 2 ** 31
    x = torch.randn(T, H, generator=g, device=dev, dtype=torch.bfloat16)
    xs = bgt.moe_gather(x, offs, pos)
    rows = torch.cat([torch.arange(100, device=dev), torch.arange(T * k - 100, T * k, device=dev),
                      torch.randint(0, T * k, (200,), generator=g, device=dev)])
    assert torch.equal(xs[rows], x[tok[rows].long()])
    w = torch.rand(T, k, generator=g, device=dev)
    y = bgt.moe_combine(xs, pos, w)
    t = torch.cat([torch.arange(100, device=dev), torch.arange(T - 100, T, device=dev)])
    ref = x[t].double() * w[t].double().sum(1, keepdim=True)
    assert ((y[t].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 8 * U) + 1e-30).all()
    dys, dw = bgt.moe_combine_backward(x, xs, offs, pos, w)
    last = int(T * k - 1)
    owner = int(tok[last])
    i = int((pos[owner] == last).nonzero()[0])
    ref = x[owner].double() * w[owner, i].double()
    assert ((dys[last].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + 1e-30).all()
    ref = (x[t].double() ** 2).sum(1)
    assert ((dw[t].double() - ref[:, None]).abs() <= (H / 32 + 32) * U * ref[:, None]).all()


def test_more_tokens_than_a_launch_has_workgroups(bgt, dev):
    # over 2^20 workgroups' worth of tokens (a workgroup a token at this length)
    T, H, E, k = (1 << 20) + 4099, 1032, 4, 1
    ids = (torch.arange(T, device=dev) * 7 % E).to(torch.int32).view(T, 1)
    offs, tok, pos = bgt.moe_sort(ids, E)
    x = (torch.arange(T, device=dev, dtype=torch.int32) % 251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    xs = bgt.moe_gather(x, offs, pos)
    assert torch.equal(xs[:, 0], x[tok.long(), 0]) and torch.equal(xs[:, -1], x[tok.long(), 0])
    w = (torch.arange(T, device=dev) % 3).float().view(T, 1)
    y = bgt.moe_combine(xs, pos, w)
    assert torch.equal(y[:, 5].float(), (x[:, 0].float() * w[:, 0]).to(torch.bfloat16).float())
    dys, dw = bgt.moe_combine_backward(x, xs, offs, pos, w)
    assert torch.equal(dys[pos[:, 0].long(), H - 1], y[:, 5])
    assert torch.equal(dw[:, 0], x[:, 0].float() ** 2 * H)      # whole numbers below 2^24 * 4: exact
    assert xs.shape[0] > 1 << 20


def test_other_stream_and_graph(bgt, dev):
    T, H, E, k = 300, 520, 8, 2
    offs, tok, pos = routing(bgt, dev, T, E, k, 11)
    xs = [torch.randn(T, H, device=dev, dtype=torch.bfloat16) for _ in range(3)]
    w = torch.rand(T, k, device=dev)
    eager = [bgt.moe_combine(bgt.moe_gather(x, offs, pos), pos, w) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [bgt.moe_combine(bgt.moe_gather(x, offs, pos), pos, w) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    buf, rows, y = xs[0].clone(), torch.empty(T * k, H, device=dev, dtype=torch.bfloat16), None
    y = torch.empty_like(buf)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        bgt.moe_gather(buf, offs, pos, xs=rows)
        bgt.moe_combine(rows, pos, w, y=y)
    for i in (1, 2, 0, 1):
        buf.copy_(xs[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])


def test_refusals(bgt, dev):
    offs, tok, pos = routing(bgt, dev, 6, 4, 2, 0)
    x = torch.randn(6, 32, device=dev)
    ys = torch.randn(12, 32, device=dev)
    w = torch.rand(6, 2, device=dev)
    with pytest.raises(ValueError):
        bgt.moe_gather(x[:5], offs, pos)
    with pytest.raises(ValueError):
        bgt.moe_gather(x.t(), offs, pos)
    with pytest.raises(TypeError):
        bgt.moe_gather(x, offs.long(), pos)
    with pytest.raises(TypeError):
        bgt.moe_gather(x.double(), offs, pos)
    with pytest.raises(ValueError):
        bgt.moe_combine(ys[:11], pos, w)
    with pytest.raises(ValueError):
        bgt.moe_combine(ys, pos, w[:, :1].contiguous())
    with pytest.raises(TypeError):
        bgt.moe_combine(ys, pos, w.half())
    with pytest.raises(TypeError):
        bgt.moe_combine_backward(x.half(), ys, offs, pos, w)
    with pytest.raises(ValueError):
        bgt.moe_combine_backward(x, ys[:, :16].contiguous(), offs, pos, w)
    with pytest.raises(bgt.BgtError):
        bgt.moe_gather(x[:1].expand(6, 32), offs, pos)
