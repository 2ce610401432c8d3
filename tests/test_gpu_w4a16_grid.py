"""Routed W4A16 products of more passes than one dimension of a grid takes."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


def test_more_passes_than_one_grid_dimension(bgt, dev):
    """256 experts of 2603 fp32 slots, 10 to a pass: 66816 passes, more than the 65535 that
    one dimension of a grid takes. Rows with one element of few bits: outputs are exact."""
    T, E, K, N = 2603, 256, 128, 16
    g = np.random.default_rng(0)
    q = g.integers(-8, 8, (E, K, N))
    s = np.exp2(g.integers(-3, 4, (E, 1, N))).astype(np.float32)
    k, v = g.integers(0, K, T), g.integers(1, 1 << 20, T).astype(np.float32)
    x = np.zeros((T, K), np.float32)
    x[np.arange(T), k] = v
    offs = torch.arange(E + 1, dtype=torch.int32, device=dev) * T
    tok = torch.arange(T, dtype=torch.int32, device=dev).flip(0).repeat(E)
    print(f"fp32 slots {T * E} of {E} experts", flush=True)
    y = bgt.w4a16_moe_gemv(torch.from_numpy(x).to(dev), offs, tok,
                           torch.stack([packed_of(bgt, dev, c) for c in q]), torch.from_numpy(s).to(dev), N)
    want = (q[:, k[::-1]] * s).astype(np.float32) * v[::-1][None, :, None]      # E x T x N
    assert torch.equal(y.view(E, T, N), torch.from_numpy(want).to(dev))
