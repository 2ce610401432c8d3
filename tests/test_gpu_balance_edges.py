"""A router's balance loss and its gradient at their edges."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")


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


# one workgroup and many; one, two, sixteen and all lanes of a wave for a token
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("others", [NAN, -INF])
@pytest.mark.parametrize("T,E", [(5, 3), (40, 8), (3000, 60), (2000, 256)])
def test_token_of_nan(bgt, dev, T, E, others, dtype):
    """A token whose logits are NaN, all of them or one among -inf, is no padding: it counts, and makes
    the loss, P and its own gradient NaN."""
    g = torch.Generator(device=dev).manual_seed(T)
    logits = torch.randn(T, E, generator=g, device=dev).to(dtype)
    ids = torch.randint(0, E, (T, 2), generator=g, device=dev, dtype=torch.int32)
    logits[1] = -INF                                            # padding
    clean = bgt.moe_balance(logits, ids)
    bad = T // 2
    logits[bad] = others
    logits[bad, E - 1] = NAN
    loss, counts, probs, tokens = bgt.moe_balance(logits, ids)
    assert int(tokens) == T - 1 == int(clean[3]) and torch.equal(counts, clean[1])
    assert bool(loss.isnan()) and bool(probs.isnan().all())
    d = bgt.moe_balance_backward(torch.ones((), device=dev), logits, counts, tokens)
    assert bool(d[bad].isnan().all()) and not bool(d[1].any())
    d[bad] = 0
    assert not bool(d.isnan().any()) and bool(d.any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [2, 8, 100])
def test_counts_of_many_ranks(bgt, dev, E, dtype):
    """Counts whose sum passes 2^31, as the sums over a job's ranks may."""
    g = torch.Generator(device=dev).manual_seed(E)
    logits = torch.randn(50, E, generator=g, device=dev).to(dtype)
    counts = torch.randint(1 << 29, (1 << 31) - 1, (E,), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    counts[0] = (1 << 31) - 1
    counts[-1] = 1 << 30
    tokens = torch.tensor([1 << 30], dtype=torch.int32, device=dev)
    got = bgt.moe_balance_backward(torch.tensor(2.0 ** 30, device=dev), logits, counts, tokens)
    p, f = torch.softmax(logits.double(), 1), counts.double() / float(counts.double().sum())
    dot = (p * f).sum(1, keepdim=True)
    ref = E * p * (f - dot)
    # softmax of E terms, the counts' sum and the dot product: at most 100 + E / 4 roundings to fp32
    bound = (100 + E / 4) * 2.0 ** -24 * E * p * (f + dot) + torch.finfo(dtype).eps / 2 * ref.abs() * 1.01 + torch.finfo(dtype).tiny
    assert bool(((got.double() - ref).abs() <= bound).all()) and bool(got.any())


@pytest.mark.parametrize("T", [61, 5000])
def test_outputs_change_in_place(bgt, dev, T):
    """A change of one output in place leaves the others as autograd has saved them."""
    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids):
            loss, counts, probs, tokens = bgt.moe_balance(logits, ids)
            ctx.save_for_backward(logits, counts, tokens)
            seen.append(probs)
            return loss

        @staticmethod
        def backward(ctx, dloss):
            return bgt.moe_balance_backward(dloss.contiguous(), *ctx.saved_tensors), None

    seen = []
    g = torch.Generator(device=dev).manual_seed(T)
    logits = torch.randn(T, 8, generator=g, device=dev).requires_grad_()
    ids = torch.randint(0, 8, (T, 2), generator=g, device=dev, dtype=torch.int32)
    Loss.apply(logits, ids).backward()
    want = logits.grad.clone()
    logits.grad = None
    loss = Loss.apply(logits, ids)
    seen[-1].mul_(0.9)                                          # a running mean, a sum over ranks
    loss.backward()
    assert torch.equal(logits.grad, want)
    outs = bgt.moe_balance(logits.detach(), ids)
    for i, t in enumerate(outs):
        rest = [u.clone() for u in outs]
        t.zero_()
        assert all(torch.equal(u, v) for j, (u, v) in enumerate(zip(outs, rest)) if j != i)
