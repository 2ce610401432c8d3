"""A router's balance loss, the experts' counts and the logits' gradient, against 64 bits."""
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


def inputs(seed, T, E, k, pad, dev, dtype):
    g = torch.Generator(device=dev).manual_seed(seed)
    logits = 2 * torch.randn(T, E, generator=g, device=dev)
    logits[torch.rand(T, generator=g, device=dev) < pad] = float("-inf")
    logits[torch.rand(T, E, generator=g, device=dev) < 0.2 * pad] = float("-inf")
    return logits.to(dtype), plain.ids_of(g, T, E, k, pad, dev)


def reference(logits, ids):
    """(loss, counts, P, T', p, f) in 64 bits."""
    v = logits.double()
    there = (v > float("-inf")).any(1)
    p = torch.zeros_like(v)
    p[there] = torch.softmax(v[there], 1)
    E = v.shape[1]
    ok = ids[(ids >= 0) & (ids < E)].long()
    c = torch.bincount(ok, minlength=E)
    n, tokens = max(1, int(c.sum())), max(1, int(there.sum()))
    f, P = c.double() / n, p.sum(0) / tokens
    return E * (f * P).sum(), c, P, int(there.sum()), p, f


def check(bgt, logits, ids, dev):
    out = bgt.moe_balance(logits, ids)
    loss, c, P, tokens, p, f = reference(logits, ids)
    T, E = logits.shape
    assert torch.equal(out[1].long(), c) and out[3].tolist() == [tokens]
    # fp32 softmax of E terms and sums of a workgroup's tokens: at most 100 + E / 4 roundings
    tol = (100 + E / 4) * 2.0 ** -24
    assert float(out[0]) == pytest.approx(float(loss), rel=tol, abs=0)
    assert bool(((out[2].double() - P).abs() <= tol * P).all())
    d = torch.tensor(1.7, device=dev)
    got = bgt.moe_balance_backward(d, logits, out[1], out[3])
    dot = (p * f).sum(1, keepdim=True)
    scale = float(d.double()) * E / max(1, tokens)
    ref = scale * p * (f - dot)
    bound = tol * scale * p * (f + dot) + torch.finfo(logits.dtype).eps / 2 * ref.abs() * 1.01 + plain.smallest(logits.dtype)
    assert got.dtype == logits.dtype and bool(((got.double() - ref).abs() <= bound).all())
    return out, got


CASES = [(1, 1, 1, 0.0), (1, 8, 2, 0.0), (61, 8, 2, 0.1), (5, 5, 5, 0.0), (257, 60, 4, 0.3), (1000, 3, 1, 0.1), (4096, 8, 2, 0.05),
         (16381, 64, 6, 0.05), (3000, 256, 8, 0.1), (777, 129, 16, 0.0), (2000, 33, 2, 0.5)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,pad", CASES)
def test_loss_and_gradient(bgt, dev, dtype, T, E, k, pad):
    logits, ids = inputs(T + E, T, E, k, pad, dev, dtype)
    a, ga = check(bgt, logits, ids, dev)
    wide = torch.cat([logits, logits], 1)[:, :E]                # rows apart
    b, gb = check(bgt, wide, ids, dev)
    for x, y in zip((*a, ga), (*b, gb)):
        assert torch.equal(x, y)                                # equal inputs, equal bits


def test_even_routing_is_one(bgt, dev):
    logits = torch.zeros(64, 8, device=dev)
    ids = (torch.arange(128, device=dev, dtype=torch.int32) % 8).view(64, 2)
    loss, counts, probs, tokens = bgt.moe_balance(logits, ids)
    assert float(loss) == 1.0 and counts.tolist() == [16] * 8 and bool((probs == 0.125).all()) and int(tokens) == 64
    assert not bool(bgt.moe_balance_backward(torch.ones((), device=dev), logits, counts, tokens).any())


@pytest.mark.parametrize("T", [3, 5000])
def test_nothing_left(bgt, dev, T):
    logits = torch.full((T, 8), float("-inf"), device=dev)
    ids = torch.full((T, 2), -1, dtype=torch.int32, device=dev)
    loss, counts, probs, tokens = bgt.moe_balance(logits, ids)
    assert float(loss) == 0 and not bool(counts.any()) and not bool(probs.any()) and int(tokens) == 0
    assert not bool(bgt.moe_balance_backward(torch.ones((), device=dev), logits, counts, tokens).ne(0).any())
    ids[0, 0] = 99                                              # outside the experts
    assert not bool(bgt.moe_balance(logits, ids)[1].any())


def test_extreme_logits(bgt, dev):
    """The type's lowest value is an ordinary logit; NaN and +inf make their token NaN, alone."""
    logits = torch.zeros(40, 8, device=dev)
    logits[0, 1:] = torch.finfo(torch.float32).min
    logits[1] = torch.finfo(torch.float32).min
    ids = (torch.arange(80, device=dev, dtype=torch.int32) % 8).view(40, 2)
    check(bgt, logits, ids, dev)
    for bad in (float("nan"), float("inf")):
        logits[7, 3] = bad
        out = bgt.moe_balance(logits, ids)
        assert bool(out[0].isnan()) and bool(out[2].isnan().all())
        d = bgt.moe_balance_backward(torch.ones((), device=dev), logits, out[1], out[3])
        assert bool(d[7].isnan().all()) and not bool(d[:7].isnan().any()) and not bool(d[8:].isnan().any())


def test_gradient_is_the_difference(bgt, dev):
    """Against central differences, in 64 bits, of the loss with the counts held."""
    logits, ids = inputs(3, 50, 7, 2, 0.0, dev, torch.float32)
    out = bgt.moe_balance(logits, ids)
    g = bgt.moe_balance_backward(torch.ones((), device=dev), logits, out[1], out[3]).double()
    gen = torch.Generator(device=dev).manual_seed(1)
    for _ in range(5):
        v = torch.randn(50, 7, generator=gen, device=dev).double() * 1e-4
        up, down = (reference(logits.double() + s * v, ids)[0] for s in (1, -1))
        # third derivatives times 1e-12, and 2^-24 of the gradient's parts
        assert float((g * v).sum()) == pytest.approx(float(up - down) / 2, rel=1e-4, abs=1e-10)


def test_parts_of_a_batch_add_up(bgt, dev):
    """Counts and tokens summed over the parts of a batch give the whole batch's gradient."""
    logits, ids = inputs(9, 900, 16, 3, 0.1, dev, torch.float32)
    whole = bgt.moe_balance(logits, ids)
    parts = [bgt.moe_balance(logits[a:b], ids[a:b]) for a, b in ((0, 300), (300, 900))]
    counts, tokens = sum(p[1] for p in parts), sum(p[3] for p in parts)
    assert torch.equal(counts, whole[1]) and torch.equal(tokens, whole[3])
    d = torch.ones((), device=dev)
    both = torch.cat([bgt.moe_balance_backward(d, logits[a:b], counts, tokens) for a, b in ((0, 300), (300, 900))])
    assert torch.equal(both, bgt.moe_balance_backward(d, logits, whole[1], whole[3]))


def test_two_streams(bgt, dev):
    """Equal bits on two streams at once, with workspaces of their own."""
    cases = [inputs(T, T, E, 2, 0.1, dev, torch.bfloat16) for T, E in ((5000, 64), (61, 8), (2000, 256))]
    ref = [bgt.moe_balance(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append([bgt.moe_balance(*c) for c in cases])
        torch.cuda.synchronize()
        for out in got:
            for a, b in zip(out, ref):
                assert all(torch.equal(u, v) for u, v in zip(a, b))
