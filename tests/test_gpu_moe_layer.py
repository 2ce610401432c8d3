"""The routing, row and product operators together, as examples/moe_layer.py uses them.

Served: both product paths against the layer computed in 64 bits from the packed
weights, within what 16-bit intermediates (and, for many tokens, 8-bit activations)
leave. Trained: output and every gradient against plain torch autograd in 64 bits.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(x, logits, gate, up, down, k):
    """The layer in the inputs' type, every expert for every token."""
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.zeros_like(logits).scatter(1, ids, torch.softmax(top, 1))
    h = torch.nn.functional.silu(torch.matmul(x, gate)) * torch.matmul(x, up)      # E x T x inner
    return (w.t()[..., None] * torch.matmul(h, down)).sum(0)


@pytest.mark.parametrize("T,bound", [(1, 0.02), (17, 0.02), (64, 0.02), (200, 0.04)])
def test_served(layer, T, bound):
    dev, E, H, I, k = torch.device("cuda"), 8, 512, 768, 2
    g = torch.Generator(device=dev).manual_seed(T)

    def w(r, c):
        return 0.05 * torch.randn(E, r, c, generator=g, device=dev)

    gate, up, down = w(H, I), w(H, I), w(I, H)
    served = layer.ServedExperts(gate, up, down, alpha=1 << 16)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device=dev)
    y = served(x, logits, k).double()

    def unpacked(name, ws):
        scale = served.parts[name][1].double().repeat_interleave(128, 1)
        v = (ws / scale.float()).double()                      # half away from zero, as the packer
        return (torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp(-7, 7) * scale

    ref = plain(x.double(), logits.double(), unpacked("gate", gate), unpacked("up", up),
                unpacked("down", down), k)
    # bf16 roundings of gate, up, their product and the experts' rows (2^-9 each, half an
    # ulp at most, independent over 768 terms), and 8-bit activations (1/254 of a row's
    # largest, twice) past 64 tokens
    assert float((y - ref).norm() / ref.norm()) < bound


def test_trained(layer):
    dev, T, E, H, I, k = torch.device("cuda"), 300, 6, 64, 96, 2
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn(T, H, generator=g, device=dev)
    params = [torch.randn(H, E, generator=g, device=dev) / 8] + \
        [0.1 * torch.randn(E, r, c, generator=g, device=dev) for r, c in ((H, I), (H, I), (I, H))]
    dy = torch.randn(T, H, generator=g, device=dev)
    ours = [p.clone().requires_grad_() for p in (x, *params)]
    y = layer.trained_layer(*ours, k)
    y.backward(dy)
    ref = [p.double().cpu().requires_grad_() for p in (x, *params)]
    z = plain(ref[0], ref[0] @ ref[1], *ref[2:], k)
    z.backward(dy.double().cpu())
    # fp32 products of up to 300 terms in a few nested sums: 1e-5 of each tensor's norm
    for a, b in [(y, z), *((p.grad, q.grad) for p, q in zip(ours, ref))]:
        assert float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm()) < 1e-5
