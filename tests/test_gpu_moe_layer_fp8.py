"""The 8-bit operators together, as examples/moe_layer.py trains with them: routing, products,
kept activations, gradients and the balance loss in one step, against the same steps in 64 bits.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp8_plain as plain  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rows8(x):
    codes, e = plain.rows(x)
    return (codes.view(x.shape[0], -1, 128) * torch.exp2(e).t()[..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]]


def weights8(w):
    codes, e = plain.weights(w)
    return (codes * torch.exp2(e).repeat_interleave(128, 0).repeat_interleave(128, 1))[:w.shape[0], :w.shape[1]]


class Experts(torch.autograd.Function):
    """rows of x for chosen experts (T x k) in 64 bits, rounded to 8 where the layer is."""

    @staticmethod
    def forward(ctx, x, ids, gate, up, down):
        ctx.save_for_backward(x, ids, gate, up, down)
        y = x.new_zeros(*ids.shape, x.shape[1])
        ctx.kept = []
        for e in range(gate.shape[0]):
            t, i = (ids == e).nonzero(as_tuple=True)
            if len(t) == 0:
                continue
            g, u = rows8(x[t]) @ weights8(gate[e]), rows8(x[t]) @ weights8(up[e])
            h = torch.nn.functional.silu(g) * u
            y[t, i] = rows8(h) @ weights8(down[e])
            ctx.kept.append((e, t, i, rows8(x[t]), rows8(g), rows8(u), rows8(h)))
        return y

    @staticmethod
    def backward(ctx, dy):
        x, ids, gate, up, down = ctx.saved_tensors
        dx, dgate, dup, ddown = (torch.zeros_like(v) for v in (x, gate, up, down))
        for e, t, i, xe, g, u, h in ctx.kept:
            d = dy[t, i]
            dh, s = rows8(d) @ weights8(down[e]).t(), torch.sigmoid(g)
            dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
            ddown[e], dgate[e], dup[e] = h.t() @ d, xe.t() @ dg, xe.t() @ du
            dx.index_add_(0, t, rows8(dg) @ weights8(gate[e]).t() + rows8(du) @ weights8(up[e]).t())
        return dx, None, dgate, dup, ddown


@pytest.mark.parametrize("T,E,H,I,k", [(1, 4, 128, 256, 2), (61, 8, 100, 130, 2), (300, 6, 256, 384, 2), (900, 3, 64, 96, 1)])
def test_step(layer, T, E, H, I, k):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(T)
    x = torch.randn(T, H, generator=g, device=dev)
    params = [torch.randn(H, E, generator=g, device=dev) / 8] + \
        [0.1 * torch.randn(E, r, c, generator=g, device=dev) for r, c in ((H, I), (H, I), (I, H))]
    dy = torch.randn(T, H, generator=g, device=dev)
    ours = [p.clone().requires_grad_() for p in (x, *params)]
    y, balance = layer.fp8_layer(*ours, k)
    ((y * dy).sum() + 3 * balance).backward()
    ref = [p.double().requires_grad_() for p in (x, *params)]
    logits = ref[0] @ ref[1]
    top, ids = torch.topk(logits, k, dim=1)
    z = (torch.softmax(top, 1)[..., None] * Experts.apply(ref[0], ids, *ref[2:])).sum(1)
    f = torch.bincount(ids.view(-1), minlength=E).double() / (T * k)
    aux = E * (f * torch.softmax(logits, 1).mean(0)).sum()
    ((z * dy.double()).sum() + 3 * aux).backward()
    assert float(balance.detach()) == pytest.approx(float(aux.detach()), rel=1e-5)
    # fp32 values are off by 1e-7 of a row's typical element, so that one in about 2e-5 (1e-7 over
    # steps of 2^-4 of the elements, the small ones' among them) goes to the next code, 2^-3 off at
    # most: sqrt(2e-5) / 8 = 6e-4 of the norm for each of up to four roundings in a row
    for a, b in [(y, z), *((p.grad, q.grad) for p, q in zip(ours, ref))]:
        assert float((a.detach().double() - b.detach()).norm()) <= 4 * 6e-4 * float(b.detach().norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_types_and_graph_free_errors(layer, dtype):
    """16-bit layers run and give gradients of their types; a second derivative is refused."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(100, 256, generator=g, device=dev).to(dtype).requires_grad_()
    router = (torch.randn(256, 4, generator=g, device=dev) / 16).requires_grad_()
    ws = [(0.05 * torch.randn(4, r, c, generator=g, device=dev)).to(dtype).requires_grad_()
          for r, c in ((256, 384), (256, 384), (384, 256))]
    y, balance = layer.fp8_layer(x, router, *ws, 2)
    assert y.dtype == dtype and balance.dtype == torch.float32
    grads = torch.autograd.grad(y.float().square().mean() + 0.01 * balance, [x, router, *ws], create_graph=True)
    for a, b in zip(grads, (x, router, *ws)):
        assert a.dtype == b.dtype and a.shape == b.shape and bool(a.isfinite().all()) and bool(a.any())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum(a.float().square().sum() for a in grads).backward()
