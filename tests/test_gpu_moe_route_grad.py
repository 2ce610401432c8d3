"""The routing gradient where ids or values are not ordinary ones.

Places whose id is outside [0, E) have no gradient, whatever their dweights hold and
wherever the id falls (a token's lanes cover up to twice E experts). With norm "chosen"
the experts not chosen have a gradient of zero, whatever the others' is.
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


@pytest.mark.parametrize("E,k", [(2, 1), (8, 2), (9, 4), (60, 6), (130, 16)])
def test_values_that_are_not_finite(bgt, dev, E, k):
    """Norm "chosen": the weights do not depend on the experts not chosen, whose gradient
    is zero whatever the chosen ones' is, and tokens do not reach each other."""
    g = np.random.default_rng(E + k)
    T = 40
    ids = distinct(g, T, E, k)
    ids[3, 1:] = -1
    v = g.standard_normal((T, E)).astype(np.float32)
    dw = g.standard_normal((T, k)).astype(np.float32)
    plain = dw.copy(), v.copy()
    odd = np.array([2, 3, 5, 7, 11, 13, 17, 39])
    dw[2, 0], dw[3, 0], dw[5, k - 1], dw[7] = np.inf, np.nan, -np.inf, np.nan
    dw[39, 0], dw[39, k - 1] = -np.inf, np.inf
    v[11, ids[11, 0]] = np.inf                     # chosen
    v[13, ids[13]] = np.inf
    v[17, ids[17, k - 1]] = np.nan
    others = np.ones((T, E + 1), bool)
    np.put_along_axis(others, np.where(ids >= 0, ids, E), False, 1)
    others = others[:, :E]
    v[others & (g.random((T, E)) < 0.2)] = np.inf  # not chosen: of no account
    v[others & (g.random((T, E)) < 0.2)] = np.nan
    fine = np.setdiff1d(np.arange(T), odd)
    for kind, dt in TYPES.items():
        print(f"routing gradient, values not finite, E={E} k={k} {kind}", flush=True)

        def call(d, l):
            return bgt.moe_route_backward(torch.from_numpy(d).to(dev), torch.from_numpy(l).to(dt).to(dev),
                                          torch.from_numpy(ids).to(dev)).cpu().double().numpy()

        got = call(dw, v)
        assert (got[others] == 0).all()
        assert np.array_equal(got[fine], call(*plain)[fine])
        # of the chosen ones the formula's: NaN where it has inf - inf, 0 * inf or NaN
        lw = np.where(others, 0.0, torch.from_numpy(v).to(dt).double().numpy())
        for t in odd:
            at = ids[t][ids[t] >= 0]
            with np.errstate(invalid="ignore"):
                e = np.exp(lw[t, at] - lw[t, at].max())
                p, d = e / e.sum(), dw[t, :len(at)].astype(np.float64)
                want = p * (d - (p * d).sum())
            assert np.array_equal(np.isnan(got[t, at]), np.isnan(want))
            assert np.array_equal(got[t, at][np.isinf(want)], want[np.isinf(want)])
