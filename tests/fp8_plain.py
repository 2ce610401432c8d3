"""8-bit floating-point rows, weights and their operators in 64 bits, for the tests.

e4m3 codes with a power of two for each block of 128 (rows) or 128 x 128 (weights); written
from the format's definition, on the inputs' device.
"""
import torch

TOP, LOW = 448.0, -117


def padded(n):
    return -(-n // 128) * 128


def e4m3(v):
    """Doubles rounded to e4m3 (3 bits below the leading one, steps of 2^-9 at least), ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40)))
    e = e + (v.abs() >= torch.exp2(e + 1)).double() - (v.abs() < torch.exp2(e)).double()
    step = torch.exp2((e - 3).clamp(min=-9))
    return torch.round(v / step) * step


def exponent(top):
    """Least e with top <= 448 * 2^e, at least LOW."""
    e = torch.floor(torch.log2(top.clamp(min=1e-300) / TOP))
    e = e - (top <= TOP * torch.exp2(e - 1)).double() + (top > TOP * torch.exp2(e)).double()
    return e.clamp(min=LOW)


def blocks(x):
    """(M, G, 128) doubles of x (M x K), zeros behind K."""
    return torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 128)).view(x.shape[0], -1, 128)


def rows(x):
    """(codes M x K' as doubles, exponents G x M) of finite rows."""
    v = blocks(x)
    e = exponent(v.abs().amax(2))
    return e4m3(v / torch.exp2(e)[..., None]).view(x.shape[0], -1), e.t()


def weights(w):
    """(codes K' x N', exponents K'/128 x N'/128) of w (K x N)."""
    K, N = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -N % 128, 0, -K % 128))
    v = v.view(v.shape[0] // 128, 128, -1, 128)
    e = exponent(v.abs().amax((1, 3)))
    return e4m3(v / torch.exp2(e)[:, None, :, None]).reshape(padded(K), padded(N)), e


def values(q, s):
    """Doubles M x K' that codes and scales of rows stand for."""
    return q.double() * s.double().repeat_interleave(128, 0).t()


def matrix(qw, sw):
    """Doubles K' x N that codes N x K' and scales K'/128 x N'/128 stand for."""
    s = sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :qw.shape[0]]
    return qw.double().t() * s


def exponents_of(s):
    """The exponents that e8m0 bytes hold, as doubles."""
    return s.view(torch.uint8).double() - 127


def same(a, b):
    """Equal values, NaN in the same places."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def product_bound(x, w, ref, dtype):
    """Elementwise bound of x.w from the 8-bit matrix instructions: of each group of at most 16
    products all but the largest may lose up to 2^-13 of that one, 15 * 2^-13 < 2^-9 of the
    group's magnitudes; fp32 sums over K (2^-23 each); the output's rounding. fp32 outputs
    come from exact products."""
    size = x.abs() @ w.abs()
    lost = x.shape[1] * 2.0 ** -23 + (0.0 if dtype == torch.float32 else 2.0 ** -9)
    return lost * size + torch.finfo(dtype).eps / 2 * (ref.abs() + lost * size) + smallest(dtype)


def smallest(dtype):
    """Half a step of the type's subnormals."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm()) if float(b.norm()) else float(a.norm())


def route(ids, E):
    """(offs, tok, expert of each sorted slot) of ids (T x k, -1: none)."""
    T, k = ids.shape
    slots = [(int(e), t * k + i) for t, r in enumerate(ids.tolist()) for i, e in enumerate(r) if 0 <= e < E]
    slots.sort()
    offs = [sum(1 for e, _ in slots if e < x) for x in range(E + 1)]
    tok = [s // k for _, s in slots] + [-1] * (T * k - len(slots))
    dev = ids.device
    return (torch.tensor(offs, dtype=torch.int32, device=dev), torch.tensor(tok, dtype=torch.int32, device=dev),
            [e for e, _ in slots])


def ids_of(g, T, E, k, drop, dev):
    """k different experts of each token, some places -1."""
    ids = torch.argsort(torch.rand(T, E, generator=g, device=dev), dim=1)[:, :k].to(torch.int32)
    gone = torch.rand(T, k, generator=g, device=dev) < drop
    return ids.masked_fill(gone, -1)
