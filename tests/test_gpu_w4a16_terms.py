"""fp32 rows of the W4A16 products to their last bits.

An fp32 element enters the products as three 16-bit terms. The sums over whole rows in
test_gpu_w4a16.py are bounded by the fp32 additions, which are larger than the third
term; here a row has one element, or two that cancel down to the third term, so that an
output is a few roundings from the exact value and every term counts.

Bound: with one code per term, a term's product with a code is exact, its product with
the scale is rounded once (U of itself; the terms have one sign), and the three are
added in two more roundings (the second U of the output, the first 2^-7 of that): 2.1 U
of the output. 3 U is taken. The third term of the elements used is at least 128 U.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


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


def packed_of(bgt, dev, q):
    """Codes q (K x N, numpy) in the library's layout."""
    K, N = q.shape
    c = (q.T & 15).reshape(N, K // 2, 2)
    canonical = (c[..., 0] | c[..., 1] << 4).astype(np.uint8).reshape(-1)
    return bgt.repack_int4_canonical(torch.from_numpy(canonical).to(dev), K, N)


def elements(g, n):
    """fp32 values whose three terms are all full ones, and the same without the third."""
    m = g.integers(0, 1 << 23, n).astype(np.uint32) | 0x8080
    bits = (g.integers(0, 2, n).astype(np.uint32) << 31) | ((g.integers(120, 135, n).astype(np.uint32)) << 23) | m
    return bits.view(np.float32), (bits & 0xFFFFFF00).view(np.float32)


def rows_and_codes(seed, M, K, N, cancel):
    """x (M x K), its two-term form, codes without zeros. Row i has one element, or an
    element and minus its first two terms at two places of one group with equal codes."""
    g = np.random.default_rng(seed)
    q = g.integers(1, 8, (K, N)) * g.choice([-1, 1], (K, N))
    x, two = np.zeros((M, K), np.float32), np.zeros((M, K), np.float32)
    v, short = elements(g, M)
    G = K // 128
    places = [g.permutation(128) + 128 * l for l in range(G)]
    for i in range(M):
        a, b = places[i % G][2 * (i // G) % 128], places[i % G][(2 * (i // G) + 1) % 128]
        x[i, a], two[i, a] = v[i], short[i]
        if cancel:
            x[i, b] = two[i, b] = -short[i]
            q[b] = q[a]
    return x, two, q


def check(y, x, two, q, s):
    W = q.astype(np.float64) * np.repeat(s.astype(np.float64), 128, 0)
    ref = x.astype(np.float64) @ W                 # one term a sum, or an exact difference: exact
    tol = 3 * U * np.abs(ref)
    assert (np.abs(two.astype(np.float64) @ W - ref) > 8 * tol).all()      # the third term shows
    bad = ~(np.abs(y.double().cpu().numpy() - ref) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs off, rows {np.unique(np.nonzero(bad)[0])}"


def scales(seed, shape):
    return (0.01 * (0.5 + np.random.default_rng(seed + 1).random(shape))).astype(np.float32)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 6, 8, 10, 11, 23])
@pytest.mark.parametrize("K,N", [(128, 16), (640, 48), (640, 16 * 601)])
@pytest.mark.parametrize("cancel", [False, True])
def test_dense(bgt, dev, M, K, N, cancel):
    print(f"fp32 terms M={M} K={K} N={N} cancel={cancel}", flush=True)
    x, two, q = rows_and_codes(M + K + N, M, K, N, cancel)
    s = scales(M, (K // 128, N))
    y = bgt.w4a16_gemv(torch.from_numpy(x).to(dev), packed_of(bgt, dev, q), torch.from_numpy(s).to(dev), N)
    check(y, x, two, q, s)


@pytest.mark.parametrize("counts", [[0, 1, 0], [3, 1, 0, 1], [1, 5, 6, 8, 10, 23], [9, 0, 7, 8]])
@pytest.mark.parametrize("N", [48, 16 * 301])
@pytest.mark.parametrize("cancel", [False, True])
def test_routed(bgt, dev, counts, N, cancel):
    print(f"fp32 terms, slots {counts} N={N} cancel={cancel}", flush=True)
    E, K, T = len(counts), 384, sum(counts)
    made = [rows_and_codes(7 * e + N, max(n, 1), K, N, cancel) for e, n in enumerate(counts)]
    s = [scales(e, (K // 128, N)) for e in range(E)]
    # token t is slot t's, in reverse order
    x = np.concatenate([m[0][:n] for m, n in zip(made, counts)])[::-1].copy()
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    tok = np.arange(T, dtype=np.int32)[::-1].copy()
    y = bgt.w4a16_moe_gemv(torch.from_numpy(x).to(dev), torch.from_numpy(offs).to(dev),
                           torch.from_numpy(tok).to(dev), torch.stack([packed_of(bgt, dev, m[2]) for m in made]),
                           torch.from_numpy(np.stack(s)).to(dev), N)
    for e, n in enumerate(counts):
        if n:
            check(y[offs[e]:offs[e + 1]], made[e][0][:n], made[e][1][:n], made[e][2], s[e])
