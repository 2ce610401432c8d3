"""Rows past the last expert's: zeroed whole, and nothing beside them touched.

The outputs lie in larger buffers at any element's alignment, with known values on both
sides; tails of no element, of less than 16 bytes, of odd counts and of many rounds.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
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


def inside(rows, H, before, dt, dev):
    """A rows x H tensor of 7 within a buffer of 7, `before` elements from its start."""
    buf = torch.full((before + rows * H + 24,), 7.0, dtype=dt, device=dev)
    return buf, buf[before:before + rows * H].view(rows, H)


def untouched(buf, before, n):
    return bool((buf[:before] == 7).all()) and bool((buf[before + n:] == 7).all())


SIZES = [(1, 1, 2, 0), (3, 1, 2, 1), (9, 1, 1, 8), (2, 3, 2, 3), (5, 7, 2, 9), (6, 8, 1, 6), (6, 8, 1, 5), (4, 9, 3, 0),
         (7, 15, 2, 13), (33, 127, 4, 100), (64, 1000, 2, 16), (50, 4096, 2, 100), (3000, 1001, 2, 7),
         (700, 4096, 2, 699)]


@pytest.mark.parametrize("T,H,k,live", SIZES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_tails(bgt, dev, T, H, k, live, kind):
    """`live` of the T*k slots have an expert."""
    print(f"tails T={T} H={H} k={k} live={live} {kind}", flush=True)
    dt, R = TYPES[kind], T * k
    g = torch.Generator(device=dev).manual_seed(T + H)
    ids = torch.full((R,), -1, dtype=torch.int32, device=dev)
    ids[torch.randperm(R, generator=g, device=dev)[:live]] = 3
    offs, tok, pos = bgt.moe_sort(ids.view(T, k), 5)
    x = torch.randn(T, H, generator=g, device=dev).to(dt)
    ys = torch.randn(R, H, generator=g, device=dev).to(dt)
    w = torch.rand(T, k, generator=g, device=dev)
    slot_w = w.view(-1)[ids == 3].double()           # slots of one expert keep their order
    want = x[tok[:live].long()].double() * slot_w[:, None]
    plain, _ = bgt.moe_combine_backward(x, ys, offs, pos, w)
    assert ((plain[:live].double() - want).abs() <= want.abs() * (HALF_ULP[kind] + 2.0 ** -24) + TINY[kind]).all()
    for before in (0, 1, 3, 8, 13):
        buf, xs = inside(R, H, before, dt, dev)
        bgt.moe_gather(x, offs, pos, xs=xs)
        assert torch.equal(xs[:live], x[tok[:live].long()])
        assert (xs[live:] == 0).all() and untouched(buf, before, R * H)
        buf, dys = inside(R, H, before, dt, dev)
        bgt.moe_combine_backward(x, ys, offs, pos, w, dys=dys)
        assert torch.equal(dys[:live], plain[:live])
        assert (dys[live:] == 0).all() and untouched(buf, before, R * H)
