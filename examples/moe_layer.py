"""A mixture-of-experts feed-forward layer on the library's operators, served and trained.

    y_t = sum_i w_ti * ((silu(x_t G_e) * (x_t U_e)) D_e),   e = ids_ti,

with the router's k experts e and weights w of each token. Served with 4-bit expert
weights: up to 64 tokens through the weight-only products of unquantized rows
(w4a16_moe_gemv), more through the W4A8 integer-scale products (quantize_act,
w4a8_moe_gemm_is). Trained with 16- or 32-bit experts: routing, gather and combine are
autograd functions over the library's forward and backward calls.

    python examples/moe_layer.py [--tokens 1 16 64 512] [--hidden 4096] [--inner 14336]
"""
import argparse
import os
import sys
import time

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_gemm_token_amd as bgt  # noqa: E402

FEW_TOKENS = 64


# ------------------------------------------------------------------------ serving
class ServedExperts:
    """E experts' gate, up (hidden -> inner) and down (inner -> hidden) matrices in 4 bits."""

    def __init__(self, gate, up, down, alpha=1024):
        self.alpha = alpha
        self.parts = {}
        for name, ws in (("gate", gate), ("up", up), ("down", down)):
            packs = [bgt.pack_weights_int4(w.float().contiguous(), alpha=alpha) for w in ws]
            self.parts[name] = tuple(torch.stack([p[key] for p in packs])
                                     for key in ("packed", "fscale", "iscale")) + (ws.shape[2],)

    def few(self, name, x, offs, tok):
        packed, fscale, _, n = self.parts[name]
        return bgt.w4a16_moe_gemv(x, offs, tok, packed, fscale, n)

    def many(self, name, x, offs, tok):
        packed, _, iscale, n = self.parts[name]
        qx, sx, _ = bgt.quantize_act(x)
        return bgt.w4a8_moe_gemm_is(qx, sx, offs, tok, packed, iscale, self.alpha, n, out_dtype=x.dtype)

    def __call__(self, x, logits, k):
        """x: tokens x hidden (fp16 or bf16); logits: the router's, tokens x experts."""
        weights, ids, offs, tok, pos = bgt.moe_route(logits, k)
        product = self.few if x.shape[0] <= FEW_TOKENS else self.many
        h = torch.nn.functional.silu(product("gate", x, offs, tok)) * product("up", x, offs, tok)
        slots = torch.arange(h.shape[0], dtype=torch.int32, device=x.device)
        return bgt.moe_combine(product("down", h, offs, slots), pos, weights)


# ----------------------------------------------------------------------- training
# The library's backward calls leave no graph: a second derivative is refused.
class Route(torch.autograd.Function):
    """logits -> (weights, ids, offs, tok, pos)"""

    @staticmethod
    def forward(ctx, logits, k):
        weights, ids, offs, tok, pos = bgt.moe_route(logits, k)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids, offs, tok, pos)
        return weights, ids, offs, tok, pos

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, *_):
        logits, ids = ctx.saved_tensors
        return bgt.moe_route_backward(dweights.contiguous(), logits, ids), None


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offs, pos):
        ctx.save_for_backward(pos)
        return bgt.moe_gather(x, offs, pos)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return bgt.moe_gather_backward(dxs.contiguous(), ctx.saved_tensors[0]), None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, offs, pos, weights):
        ctx.save_for_backward(ys, offs, pos, weights)
        return bgt.moe_combine(ys, pos, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, offs, pos, weights = ctx.saved_tensors
        dys, dweights = bgt.moe_combine_backward(dy.contiguous(), ys, offs, pos, weights)
        return dys, None, None, dweights


def trained_layer(x, router, gate, up, down, k):
    """The layer's output for training: router hidden x experts; gate, up, down as in
    ServedExperts, in x's type."""
    logits = x.float() @ router
    weights, _, offs, _, pos = Route.apply(logits, k)
    xs = Gather.apply(x, offs, pos)
    ys = []
    for e, n in enumerate((offs[1:] - offs[:-1]).tolist()):
        rows = xs[sum(y.shape[0] for y in ys):][:n]
        ys.append((torch.nn.functional.silu(rows @ gate[e]) * (rows @ up[e])) @ down[e])
    ys.append(xs.new_zeros(xs.shape[0] - sum(y.shape[0] for y in ys), x.shape[1]))
    return Combine.apply(torch.cat(ys), offs, pos, weights)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, nargs="*", default=[1, 16, 64, 512])
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    a = ap.parse_args()
    torch.manual_seed(0)
    dev = torch.device("cuda")
    E, H, I = a.experts, a.hidden, a.inner

    def experts(rows, cols, dtype):
        return (0.02 * torch.randn(E, rows, cols, device=dev)).to(dtype)

    served = ServedExperts(experts(H, I, torch.bfloat16), experts(H, I, torch.bfloat16),
                           experts(I, H, torch.bfloat16))
    router = torch.randn(H, E, device=dev) / H ** 0.5
    for T in a.tokens:
        x = torch.randn(T, H, device=dev, dtype=torch.bfloat16)
        logits = x.float() @ router
        for _ in range(3):
            y = served(x, logits, a.topk)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            y = served(x, logits, a.topk)
        torch.cuda.synchronize()
        print("serve %4d tokens: %8.1f us, |y| %.3f" % (T, (time.perf_counter() - t) / 20 * 1e6,
                                                        float(y.float().norm())), flush=True)

    h, i = 256, 512                                  # a small layer, a few steps
    params = [torch.nn.Parameter(p) for p in (torch.randn(h, E, device=dev) / h ** 0.5,
              *(0.05 * torch.randn(E, r, c, device=dev) for r, c in ((h, i), (h, i), (i, h))))]
    opt = torch.optim.Adam(params, lr=3e-3)
    x, goal = torch.randn(1000, h, device=dev), torch.randn(1000, h, device=dev)
    for step in range(5):
        loss = (trained_layer(x, *params, a.topk) - goal).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print("train step %d: loss %.4f" % (step, float(loss.detach())), flush=True)


if __name__ == "__main__":
    main()
