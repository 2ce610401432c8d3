"""The example layer's autograd functions refuse a second derivative (no GPU needed).

Their backward calls are the library's and leave no graph, so a second derivative
would silently lack their terms. The library's calls are replaced by torch forms
outside the graph.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Plain:
    """The library's calls on the CPU, one expert a token, token t in slot t."""

    @staticmethod
    @torch.no_grad()
    def moe_route(logits, k):
        ids = torch.topk(logits, k, dim=1)[1].to(torch.int32)
        pos = torch.arange(ids.numel(), dtype=torch.int32).view(ids.shape)
        lists = [torch.zeros(n, dtype=torch.int32) for n in (logits.shape[1] + 1, ids.numel())]
        return torch.softmax(logits, 1).gather(1, ids.long()), ids, *lists, pos

    @staticmethod
    @torch.no_grad()
    def moe_route_backward(dweights, logits, ids):
        return logits * dweights.sum()

    @staticmethod
    @torch.no_grad()
    def moe_gather(x, offs, pos):
        return x[pos.view(-1).long()].clone()

    @staticmethod
    @torch.no_grad()
    def moe_gather_backward(dxs, pos):
        return dxs[pos.view(-1).long()].clone()

    @staticmethod
    @torch.no_grad()
    def moe_combine(ys, pos, weights):
        return weights * ys[pos.view(-1).long()]

    @staticmethod
    @torch.no_grad()
    def moe_combine_backward(dy, ys, offs, pos, weights):
        return weights * dy, (ys * dy).sum(1, keepdim=True)


@pytest.fixture()
def layer(monkeypatch):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "bgt", Plain)
    return m


def first_and_second(f, x):
    """A second derivative of f(x) + x^3, whose own part torch can give."""
    first, = torch.autograd.grad(f(x) + (x ** 3).sum(), x, create_graph=True)
    assert torch.isfinite(first).all()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.sum().backward()


def test_second_derivatives_are_refused(layer):
    T, H = 5, 3
    x = torch.randn(T, H, requires_grad=True)
    pos = torch.arange(T, dtype=torch.int32).view(T, 1)
    offs = torch.tensor([0, T], dtype=torch.int32)
    w = torch.rand(T, 1, requires_grad=True)
    first_and_second(lambda a: (layer.Gather.apply(a, offs, pos) ** 2).sum(), x)
    first_and_second(lambda a: (layer.Combine.apply(a, offs, pos, w) ** 2).sum(), x)
    first_and_second(lambda a: (layer.Combine.apply(x, offs, pos, a) ** 2).sum(), w)
    logits = torch.randn(T, H, requires_grad=True)
    first_and_second(lambda a: (layer.Route.apply(a, 1)[0] ** 2).sum(), logits)
