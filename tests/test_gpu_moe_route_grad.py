"""The routing gradient where ids or values are not ordinary ones.

Places whose id is outside [0, E) have no gradient, whatever their dweights hold and
wherever the id falls (a token's lanes cover up to twice E experts).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
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


def distinct(g, T, E, k):
    return np.argsort(g.random((T, E)), axis=1)[:, :k].astype(np.int32)


def gradient(v, ids, dw, norm):
    """dl (T x E) in 64 bits and the size of its terms; ids outside [0, E) are skipped."""
    T, E = v.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, E)
    mask = np.zeros((T, E + 1), bool)
    np.put_along_axis(mask, at, True, 1)
    d = np.zeros((T, E + 1))
    np.put_along_axis(d, at, np.where(ok, dw, 0.0).astype(np.float64), 1)
    d, base = d[:, :E], v if norm == "all" else np.where(mask[:, :E], v, -np.inf)
    m = base.max(1, keepdims=True)
    e = np.exp(base - np.where(m == -np.inf, 0.0, m))
    s = e.sum(1, keepdims=True)
    p = np.divide(e, s, out=np.zeros_like(e), where=s != 0)
    return p * (d - (p * d).sum(1, keepdims=True)), p * (np.abs(d) + (p * np.abs(d)).sum(1, keepdims=True))


@pytest.mark.parametrize("E", [1, 3, 5, 9, 20, 33, 60, 65, 130, 200, 256])
@pytest.mark.parametrize("norm", ["chosen", "all"])
def test_ids_outside(bgt, dev, E, norm):
    k = min(E, 6)
    g = np.random.default_rng(E)
    full = 4 if E <= 8 else 8                      # experts that a token's lanes go up to, and past
    outside = np.array([-1, -2, E, E + 1, E + 2, E + full, 2 * E - 1, 2 * E, 255, 256, 1000, -2 ** 31, 2 ** 31 - 1])
    outside = outside[(outside < 0) | (outside >= E)]
    T = 4 * len(outside)
    ids = distinct(g, T, E, k)
    dw = g.standard_normal((T, k)).astype(np.float32)
    gone = g.random((T, k)) < 0.3
    gone[np.arange(T), np.arange(T) % k] = True    # every value of `outside` in some place
    gone[T - 1] = True                             # and a token with no place left
    ids[gone] = outside[(np.arange(T)[:, None] + np.zeros(k, int)) % len(outside)][gone]
    dw[gone] = np.array([np.nan, np.inf, -np.inf, 1e30], np.float32)[g.integers(0, 4, int(gone.sum()))]
    for kind, dt in TYPES.items():
        print(f"routing gradient with ids outside, E={E} {kind} {norm}", flush=True)
        logits = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).to(dt)
        got = bgt.moe_route_backward(torch.from_numpy(dw).to(dev), logits.to(dev),
                                     torch.from_numpy(ids).to(dev), norm=norm)
        same = bgt.moe_route_backward(torch.from_numpy(np.where(gone, np.float32(0), dw)).to(dev), logits.to(dev),
                                      torch.from_numpy(np.where(gone, np.int32(-1), ids)).to(dev), norm=norm)
        assert torch.equal(got, same)
        want, size = gradient(logits.double().numpy(), ids, dw, norm)
        # p: the exponential and a sum and a division in fp32, logits within 12 of the largest;
        # the inner sum over a tree of depth at most 12, two more operations
        tol = size * 160 * U + np.abs(want) * HALF_ULP[kind] + (6e-8 if kind == "f16" else 1e-37)
        assert (np.abs(got.cpu().double().numpy() - want) <= tol).all()
