"""Routing of a mixture-of-experts layer against plain 64-bit computations.

Expert choices, sorted slots, offsets and positions must be equal; weights and
gradients lie within bounds derived from the operations in fp32. Sizes cover
one token to tens of thousands, every expert count at which the kernels change
their lane layout, ties, masks that leave a token few experts or none, masks
of the type's lowest value, infinities and NaN.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24          # half an ulp of fp32, relative
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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


def choose(v, k):
    """ids of the k largest of each row (float64 numpy): ties to the lower index,
    NaN and -inf never."""
    key = np.where(np.isnan(v), -np.inf, v)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(key, order, 1)
    return np.where(top > -np.inf, order, -1).astype(np.int32)


def softmax(v, ids, norm):
    """p (T x E) over the chosen experts or over all, in 64 bits."""
    T, E = v.shape
    mask = np.zeros((T, E + 1), bool)
    np.put_along_axis(mask, np.where(ids >= 0, ids, E), True, 1)
    base = v if norm == "all" else np.where(mask[:, :E], v, -np.inf)
    m = np.max(np.where(np.isnan(base), -np.inf, base), axis=1, keepdims=True)
    m = np.where(m == -np.inf, 0.0, m)
    with np.errstate(invalid="ignore"):
        e = np.exp(base - m)
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0), m


def sort_slots(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    n = int(ok.sum())
    offs = np.zeros(E + 1, np.int32)
    offs[1:] = np.cumsum(np.bincount(flat[ok], minlength=E))
    tok = np.full(T * k, -1, np.int32)
    tok[:n] = order[:n] // k
    pos = np.full(T * k, -1, np.int32)
    pos[order[:n]] = np.arange(n)
    return offs, tok, pos.reshape(T, k)


def logits_of(seed, T, E, kind, pad=0.0, ties=False):
    g = np.random.default_rng(seed)
    v = g.standard_normal((T, E)).astype(np.float32) + 0.5 * g.standard_normal(E).astype(np.float32)
    if ties:
        v = np.round(v * 2) / 2
    if pad:
        v[g.random(T) < pad] = -np.inf
        v[g.random((T, E)) < 0.2] = -np.inf
    return torch.from_numpy(v).to(TYPES[kind])


def check_route(bgt, logits, k, norm, out):
    w, ids, offs, tok, pos = [t.cpu().numpy() for t in out]
    v = logits.cpu().double().numpy()
    E = v.shape[1]
    want = choose(v, k)
    np.testing.assert_array_equal(ids, want)
    for got, ref in zip((offs, tok, pos), sort_slots(want, E)):
        np.testing.assert_array_equal(got, ref)
    p, m = softmax(v, want, norm)
    at = np.clip(want, 0, None)
    pw = np.where(want >= 0, np.take_along_axis(p, at, 1), 0.0)
    # exp of a difference rounded once (|l - m| U), exp itself and the sum of at
    # most 256 terms in a tree of depth at most 12 (each at most 2 ulp), one division
    far = np.abs(np.take_along_axis(np.where(np.isfinite(v), v, 0.0), at, 1) - m)
    tol = pw * (far + 48) * 2 * U + 1e-37
    fine = ~np.isnan(pw)
    np.testing.assert_array_equal(np.isnan(w), ~fine)
    assert (np.abs(w - pw)[fine] <= tol[fine]).all()


ROUTES = [(1, 8, 2), (1, 1, 1), (2, 3, 3), (7, 8, 8), (64, 9, 4), (63, 16, 2), (65, 17, 16),
          (255, 32, 6), (256, 33, 5), (257, 60, 4), (100, 64, 8), (1000, 65, 8), (513, 128, 8),
          (300, 129, 3), (77, 256, 8), (4096, 8, 2), (4097, 8, 1), (16381, 64, 6), (40000, 8, 2)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route(bgt, dev, T, E, k, norm):
    for kind in TYPES:
        say(f"route T={T} E={E} k={k} {kind} {norm}")
        logits = logits_of(T + E * 7 + k, T, E, kind, ties=kind == "f16").to(dev)
        check_route(bgt, logits, k, norm, bgt.moe_route(logits, k, norm=norm))


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (40, 8, 2), (333, 64, 8), (5000, 20, 4), (9000, 200, 3)])
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route_masks(bgt, dev, T, E, k, norm):
    # whole tokens masked, single experts masked: fewer than k left, or none
    for kind in TYPES:
        say(f"route masked T={T} E={E} k={k} {kind} {norm}")
        logits = logits_of(T + E + k, T, E, kind, pad=0.3)
        logits[0] = -np.inf
        logits[T // 2, 1:] = -np.inf
        logits = logits.to(dev)
        check_route(bgt, logits, k, norm, bgt.moe_route(logits, k, norm=norm))


def test_route_all_masked(bgt, dev):
    logits = torch.full((50, 8), -np.inf, device=dev)
    w, ids, offs, tok, pos = bgt.moe_route(logits, 2)
    assert (w == 0).all() and (ids == -1).all() and (offs == 0).all()
    assert (tok == -1).all() and (pos == -1).all()


@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route_lowest_value_infinities_nan(bgt, dev, norm):
    for kind, dt in TYPES.items():
        low = torch.finfo(dt).min
        v = logits_of(3, 12, 8, kind)
        v[0] = low                       # the type's lowest value is a value like any other
        v[1, 2:] = low
        v[2, 0] = np.inf                 # its row's weights are NaN, its expert is chosen first
        v[3, 4] = np.nan                 # never chosen; NaN weights only where all are summed
        v[4] = np.nan
        v[5, 1:] = np.nan
        v[6] = torch.finfo(dt).max
        say(f"route special {kind} {norm}")
        check_route(bgt, v.to(dev), 3, norm, bgt.moe_route(v.to(dev), 3, norm=norm))


def test_route_strides_and_outputs_given(bgt, dev):
    full = torch.randn(70, 40, device=dev)
    view = full[:, 3:23]                 # row stride 40, base 12 bytes into a row
    check_route(bgt, view, 4, "all", bgt.moe_route(view, 4, norm="all"))
    half = full.to(torch.bfloat16)[::2, 1:18]
    check_route(bgt, half, 2, "chosen", bgt.moe_route(half, 2))
    one = full[5:6, 3:23]
    check_route(bgt, one, 4, "chosen", bgt.moe_route(one, 4))
    w = torch.full((70, 4), -5.0, device=dev)
    out = bgt.moe_route(view, 4, weights=w)
    assert out[0] is w
    check_route(bgt, view, 4, "chosen", out)


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (33, 8, 2), (1024, 8, 2), (1025, 256, 16), (3000, 5, 4),
                                   (16384, 60, 8), (70001, 128, 1), (400000, 8, 2)])
def test_sort(bgt, dev, T, E, k):
    say(f"sort T={T} E={E} k={k}")
    g = np.random.default_rng(T + E)
    ids = g.integers(-1, E + 1, (T, k)).astype(np.int32)     # -1 and E: dropped
    ids[g.random((T, k)) < 0.3] = E // 2                     # a busy expert
    got = bgt.moe_sort(torch.from_numpy(ids).to(dev), E)
    for a, b in zip(got, sort_slots(ids, E)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (9, 3, 3), (100, 16, 4), (257, 33, 5), (100, 64, 8),
                                   (301, 128, 8), (65, 256, 16), (8191, 60, 4)])
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route_backward(bgt, dev, T, E, k, norm):
    for kind in TYPES:
        say(f"route backward T={T} E={E} k={k} {kind} {norm}")
        logits = logits_of(T + E, T, E, kind, pad=0.1 if T > 9 else 0.0)
        v = logits.double().numpy()
        ids = choose(v, k)
        dw = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
        got = bgt.moe_route_backward(torch.from_numpy(dw).to(dev), logits.to(dev),
                                     torch.from_numpy(ids).to(dev), norm=norm)
        assert got.dtype == logits.dtype and got.shape == logits.shape
        p, m = softmax(v, ids, norm)
        d = np.zeros((T, E + 1))
        np.put_along_axis(d, np.where(ids >= 0, ids, E), dw.astype(np.float64), 1)
        d = d[:, :E]
        want = p * (d - (p * d).sum(1, keepdims=True))
        # p as in the forward bound (logits within 12 of the largest or negligible),
        # the inner sum over a tree of depth at most 12, two more operations
        size = p * (np.abs(d) + (p * np.abs(d)).sum(1, keepdims=True))
        tol = size * 160 * U + np.abs(want) * HALF_ULP[kind] + (6e-8 if kind == "f16" else 1e-37)
        assert (np.abs(got.cpu().double().numpy() - want) <= tol).all()


@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_route_backward_against_differences(bgt, dev, norm):
    # the forward call's weights on both sides of each logit: f = sum(c * w)
    T, E, k, h = 6, 9, 3, 2.0 ** -7
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(T, E, generator=g)
    c = torch.randn(T, k, generator=g)
    _, ids, *_ = bgt.moe_route(logits.to(dev), k, norm=norm)
    got = bgt.moe_route_backward(c.to(dev), logits.to(dev), ids, norm=norm).cpu().double()

    def f(v):
        w, i, *_ = bgt.moe_route(v.to(dev), k, norm=norm)
        assert torch.equal(i, ids)                 # the choice does not change at these steps
        return (w.cpu().double() * c.double()).sum(1)

    for e in range(E):
        step = torch.zeros(T, E)
        step[:, e] = h
        diff = (f(logits + step) - f(logits - step)) / (2 * h)
        # third derivative of a softmax output is at most 1 in size; weights carry
        # a few U, divided by the step
        tol = c.abs().double().sum(1) * (h * h / 6 + 64 * U / h)
        assert ((got[:, e] - diff).abs() <= tol).all()


def test_route_other_stream_and_graph(bgt, dev):
    logits = [logits_of(i, 700, 8, "bf16", pad=0.1).to(dev) for i in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [bgt.moe_route(v, 2) for v in logits]
    side.synchronize()
    for v, o in zip(logits, outs):
        check_route(bgt, v, 2, "chosen", o)
    buf = logits[0].clone()
    out = bgt.moe_route(buf, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bgt.moe_route(buf, 2, weights=out[0], ids=out[1], offs=out[2], tok=out[3], pos=out[4])
    for v in (logits[1], logits[2], logits[0], logits[1]):
        buf.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_route(bgt, v, 2, "chosen", out)


def test_route_refusals(bgt, dev):
    v = torch.randn(4, 8, device=dev)
    for k in (0, 9, -1):
        with pytest.raises(bgt.BgtError) as e:
            bgt.moe_route(v, k)
        assert e.value.status == bgt.BGT_ERR_SHAPE
    with pytest.raises(bgt.BgtError):
        bgt.moe_route(torch.randn(4, 20, device=dev), 17)
    with pytest.raises(bgt.BgtError):
        bgt.moe_route(torch.randn(4, 257, device=dev), 2)
    with pytest.raises(bgt.BgtError):
        bgt.moe_route(torch.empty(0, 8, device=dev), 2)
    with pytest.raises(bgt.BgtError):
        bgt.moe_route(v[:1].expand(4, 8), 2)       # rows on top of each other
    with pytest.raises(ValueError):
        bgt.moe_route(v, 2, norm="sigmoid")
    with pytest.raises(ValueError):
        bgt.moe_route(v.t(), 2)
    with pytest.raises(ValueError):
        bgt.moe_route(v.cpu(), 2)
    with pytest.raises(TypeError):
        bgt.moe_route(v.double(), 2)
    with pytest.raises(TypeError):
        bgt.moe_sort(torch.zeros(4, 2, dtype=torch.int64, device=dev), 8)
    with pytest.raises(ValueError):
        bgt.moe_route_backward(torch.zeros(4, 3, device=dev), v,
                               torch.zeros(4, 2, dtype=torch.int32, device=dev))
