"""Measured cases of the 8-bit floating-point operators of training and serving, and of the
router's balance loss.

    store     activations or weights held in 8 bits (e4m3) with a power of two for each block:
              rows in blocks of 128 and back, weights in blocks of 128 x 128 in both
              directions of the product, silu(g) * u with g and u kept in 8 bits; "gate_grad"
              is the latter's gradient from what was kept
    linear    rows stored in 8 bits times such a weight matrix; "grad": a gradient's rows times
              the matrix turned
    experts   the same for routed slots, each times its own expert's matrix
    wgrad     a weight's gradient from the rows kept in 8 bits, of one matrix or of every expert
    balance   a router's balance loss with the experts' counts; "grad": also the logits' gradient

`run` computes each operator either in elementary torch operations, in 32 bits and rounded
once at the end, or (`own`) through bit_gemm_token_amd. Sizes are those of the repository's
benchmark (4096, 11008, 14336, 22016; 8 experts, 2 for each token) and generic ones.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
TOP = 448.0                      # the largest e4m3 value
LOW = -117                       # the smallest exponent of a block's scale


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a training step's weights of one layer, stored for both directions of the product
        dict(name="store_weights", op="store", what="weights", K=4096, N=14336, type="bf16"),
        # a training batch through the gate of a feed-forward layer, gate and up kept in 8 bits
        dict(name="store_gate", op="store", what="gate", M=8192, K=14336, type="bf16"),
        # its gradient at odd sizes, in fp32
        dict(name="store_gate_grad", op="store", what="gate_grad", M=1021, K=11000, type="f32"),
        # one token through an attention projection: latency
        dict(name="linear_one", op="linear", M=1, K=4096, N=4096, type="bf16", grad=False),
        # a decode batch (odd count) times the widest layer of the benchmark
        dict(name="linear_batch", op="linear", M=61, K=4096, N=22016, type="f16", grad=False),
        # a training batch's gradient through an up projection
        dict(name="linear_train", op="linear", M=8192, K=4096, N=14336, type="bf16", grad=True),
        # a decode batch through two of eight experts' up projections
        dict(name="experts_decode", op="experts", T=16, E=8, k=2, K=4096, N=14336, type="bf16", pad=0.0, grad=False),
        # a training batch through the experts, some of its tokens padding that no expert takes
        dict(name="experts_train", op="experts", T=4096, E=8, k=2, K=4096, N=14336, type="bf16", pad=0.05, grad=False),
        # gradient of one projection's weights from a long sequence
        dict(name="wgrad_layer", op="wgrad", M=8191, K=4096, N=4096, E=0, type="bf16"),
        # gradients of every expert's weights, many small experts, fp32
        dict(name="wgrad_experts", op="wgrad", M=2048, K=1024, N=1408, E=32, k=4, type="f32", pad=0.1),
        # a small batch's balance loss
        dict(name="balance_few", op="balance", T=61, E=8, k=2, type="f32", pad=0.0, grad=False),
        # a training batch over many small experts, with the router's gradient
        dict(name="balance_train", op="balance", T=16381, E=64, k=6, type="bf16", pad=0.05, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 128, as layers' widths are, some of 8, a few of any size."""
    n, p = _log(rng, lo, hi), rng.random()
    return max(128, n // 128 * 128) if p < 0.7 else max(8, n // 8 * 8) if p < 0.9 else n


def draw(rng):
    op = rng.choice(["store", "linear", "experts", "wgrad", "balance"])
    kind = rng.choice(["f32", "f16", "bf16"])
    K, N = _width(rng, 64, 14336), _width(rng, 64, 22016)
    if op == "store":
        what = rng.choice(["rows", "weights", "gate", "gate_grad"])
        if what == "weights":
            return dict(op=op, what=what, K=K, N=N, type=kind)
        return dict(op=op, what=what, M=min(_log(rng, 1, 8192), (1 << 26) // K), K=K, type=kind)
    if op == "linear":
        M = min(_log(rng, 1, 8192), max(1, (1 << 38) // (K * N)))
        return dict(op=op, M=M, K=K, N=N, type=kind, grad=rng.random() < 0.5)
    if op == "balance":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)), type=kind,
                    pad=rng.choice([0.0, 0.05, 0.3]), grad=rng.random() < 0.5)
    if op == "wgrad" and rng.random() < 0.5:
        N = max(8, min(N, (1 << 26) // K))
        return dict(op=op, M=min(_log(rng, 1, 8192), (1 << 37) // (K * N)), K=K, N=N, E=0, type=kind)
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    K = min(K, 4096)
    N = max(64, min(N, (8 * 4096 * 14336 if op == "experts" else 1 << 27) // (E * K)))
    T = max(1, min(_log(rng, 1, 4096), (1 << 38) // (k * K * N)))
    pad = rng.choice([0.0, 0.1])
    if op == "experts":
        return dict(op=op, T=T, E=E, k=k, K=K, N=N, type=kind, pad=pad, grad=rng.random() < 0.3)
    return dict(op=op, M=T, K=K, N=N, E=E, k=k, type=kind, pad=pad)


# ------------------------------------------------------------------------ inputs
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _activations(g, M, K, dev):
    """Normal rows with one channel in a hundred twenty times as large."""
    x = torch.randn(M, K, generator=g, device=dev)
    x[:, torch.randperm(K, generator=g, device=dev)[: max(1, K // 100)]] *= 20
    return x


def _gradients(g, M, K, dev):
    """Gradients' rows: small, of sizes that differ by an order of magnitude between rows."""
    size = torch.exp(torch.randn(M, 1, generator=g, device=dev))
    return 1e-3 * size * torch.randn(M, K, generator=g, device=dev)


def _weights(g, K, N, dev):
    w = 0.02 * torch.randn(K, N, generator=g, device=dev)
    w[torch.rand(K, N, generator=g, device=dev) < 0.001] *= 10
    return w


def _logits(g, T, E, pad, dev):
    """Normal logits with a bias per expert, as trained routers give; of a padding
    token every logit is -inf, and a few other entries are masked too."""
    logits = torch.randn(T, E, generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
    if pad:
        gone = torch.rand(T, 1, generator=g, device=dev) < pad
        some = torch.rand(T, E, generator=g, device=dev) < 0.1 * pad
        logits = logits.masked_fill(gone | some, -math.inf)
    return logits


def _choose(logits, k):
    """The k largest logits of each row, -1 where too few are left."""
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    return ids[:, :k].masked_fill(top[:, :k] == -math.inf, -1).to(torch.int32)


def _sorted(ids, E):
    """(offs, tok): slots sorted by expert, tokens in order within an expert."""
    T, k = ids.shape
    key = torch.where(ids < 0, E, ids.long()).view(-1)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offs = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offs, (order // k).masked_fill(key[order] == E, -1).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, dt = case, TYPES[case["type"]]
    s = {"case": dict(case)}
    if c["op"] == "store":
        if c["what"] == "weights":
            s["w"] = _weights(g, c["K"], c["N"], dev).to(dt)
        elif c["what"] == "rows":
            s["x"] = _activations(g, c["M"], c["K"], dev).to(dt)
        else:
            gate, up = (_activations(g, c["M"], c["K"], dev).to(dt) for _ in range(2))
            if c["what"] == "gate":
                s["gate"], s["up"] = gate, up
            else:                                   # what the forward pass has kept
                s["kept"] = (*_store(gate), *_store(up))
                s["dh"] = _gradients(g, c["M"], c["K"], dev).to(dt)
        return s
    if c["op"] == "linear":
        # the product runs over K into N, of a gradient over N into K
        over = c["N"] if c["grad"] else c["K"]
        s["x"] = (_gradients if c["grad"] else _activations)(g, c["M"], over, dev).to(dt)
        q, scale, qt, scale_t = _store_weights(_weights(g, c["K"], c["N"], dev).to(dt))
        s["qw"], s["sw"] = (qt, scale_t) if c["grad"] else (q, scale)
        return s
    if c["op"] == "wgrad" and c["E"] == 0:
        s["qx"], s["sx"] = _store(_activations(g, c["M"], c["K"], dev).to(dt))
        s["dy"] = _gradients(g, c["M"], c["N"], dev).to(dt)
        return s
    T = c["M"] if c["op"] == "wgrad" else c["T"]
    logits = _logits(g, T, c["E"], c["pad"], dev)
    ids = _choose(logits, c["k"])
    if c["op"] == "balance":
        s["logits"], s["ids"] = logits.to(dt), ids
        s["dloss"] = torch.rand((), generator=g, device=dev)
        return s
    # the routing that such a program already holds, and the most slots of an expert
    s["offs"], s["tok"] = _sorted(ids, c["E"])
    s["most"] = max(1, int((s["offs"][1:] - s["offs"][:-1]).max()))
    if c["op"] == "wgrad":
        s["qx"], s["sx"] = _store(_activations(g, T, c["K"], dev).to(dt))
        s["dy"] = _gradients(g, T * c["k"], c["N"], dev).to(dt)
        return s
    over = c["N"] if c["grad"] else c["K"]
    s["x"] = (_gradients if c["grad"] else _activations)(g, T, over, dev).to(dt)
    both = [_store_weights(_weights(g, c["K"], c["N"], dev).to(dt))[2 * c["grad"]:][:2] for _ in range(c["E"])]
    s["qw"] = torch.stack([q.view(torch.uint8) for q, _ in both]).view(torch.float8_e4m3fn)
    s["sw"] = torch.stack([v.view(torch.uint8) for _, v in both]).view(torch.float8_e8m0fnu)
    return s


# ------------------------------------------------------------------- plain forms
def _exponents(top):
    """The least e with top <= 448 * 2^e, but at least LOW (top finite, fp32)."""
    bits = top.view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp(min=LOW)


def _power(e):
    """2^e as fp32, e in the normal range."""
    return ((e + 127) << 23).view(torch.float32)


def _bytes(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _store(x):
    """Rows in 8 bits: values M x K' (K' = K up to a multiple of 128, zeros behind) and
    the blocks' scales, K'/128 x M."""
    M, K = x.shape
    G = _blocks(K)
    v = torch.zeros(M, G * BLOCK, device=x.device)
    v[:, :K] = x.float()
    v = v.view(M, G, BLOCK)
    e = _exponents(v.abs().amax(2))
    q = (v * _power(-e)[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.view(M, G * BLOCK), _bytes(e.t().contiguous())


def _rows(q, scale, K):
    """The rows that values and scales stand for, in fp32."""
    return (q.float() * scale.float().t().repeat_interleave(BLOCK, 1))[:, :K]


def _store_weights(w):
    """K x N weights in 8 bits: N x K' values and K'/128 x N'/128 scales for the product over
    K, and K x N' values and the scales turned for the one over N."""
    K, N = w.shape
    A, B = _blocks(K), _blocks(N)
    v = torch.zeros(A * BLOCK, B * BLOCK, device=w.device)
    v[:K, :N] = w.float()
    v = v.view(A, BLOCK, B, BLOCK)
    e = _exponents(v.abs().amax((1, 3)))
    q = (v * _power(-e)[:, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(A * BLOCK, B * BLOCK)
    turned = q.view(torch.uint8).t()[:N].contiguous().view(torch.float8_e4m3fn)
    return turned, _bytes(e), q[:K].contiguous(), _bytes(e.t().contiguous())


def _matrix(q, scale):
    """The weights that values (.. x N x K') and scales (.. x K'/128 x N'/128) stand for, in
    fp32, K' x N."""
    w = q.float().transpose(-1, -2)
    s = scale.float().repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)
    return (w * s[..., :w.shape[-1]]).contiguous()


def _padded(q, scale):
    return _rows(q, scale, q.shape[1])


def _place(offs, R):
    """Of each slot: its expert, whether it has one, and its place within the expert."""
    r = torch.arange(R, device=offs.device)
    e = (r[:, None] >= offs[None, 1:]).sum(1)
    there = e < offs.numel() - 1
    e = e.clamp(max=offs.numel() - 2)
    return e, there, r - offs[e]


def _by_expert(rows, e, there, at, E, most):
    """Slots' rows as E x most x H, zeros in places without a slot."""
    full = rows.new_zeros(E, most, rows.shape[1])
    return full.index_put_((e, at.clamp(max=most - 1)), torch.where(there[:, None], rows, 0.0), accumulate=True)


def _experts(s):
    x, offs, tok = s["x"], s["offs"], s["tok"]
    q, scale = _store(x)
    e, there, at = _place(offs, tok.numel())
    rows = _padded(q, scale)[tok.clamp(min=0).long()]
    full = _by_expert(rows, e, there, at, offs.numel() - 1, s["most"])
    y = torch.bmm(full, _matrix(s["qw"], s["sw"]))[e, at.clamp(max=s["most"] - 1)]
    return q, scale, torch.where(there[:, None], y, 0.0).to(x.dtype)


def _balance(s):
    c = s["case"]
    v, ids = s["logits"].float(), s["ids"]
    E = v.shape[1]
    some = (v > -math.inf).any(1, keepdim=True)
    p = torch.exp(v - torch.where(some, v.amax(1, keepdim=True), 0.0))
    p = torch.where(some, p / p.sum(1, keepdim=True).clamp(min=1e-30), 0.0)
    counts = (ids.view(-1, 1) == torch.arange(E, device=v.device)).sum(0)
    tokens = some.sum()
    f = counts.float() / counts.sum().clamp(min=1)
    mean = (p.double().sum(0) / tokens.clamp(min=1)).float()
    loss = E * (f * mean).sum()
    out = (loss, counts.to(torch.int32), mean, tokens.to(torch.int32).view(1))
    if not c["grad"]:
        return out
    d = s["dloss"] * E / tokens.clamp(min=1) * p * (f - (p * f).sum(1, keepdim=True))
    return *out, d.to(s["logits"].dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "balance":
        return _balance(s)
    if c["op"] == "experts":
        return _experts(s)
    if c["op"] == "linear":
        q, scale = _store(s["x"])
        return q, scale, (_padded(q, scale) @ _matrix(s["qw"], s["sw"])).to(s["x"].dtype)
    if c["op"] == "wgrad":
        x, dy = _rows(s["qx"], s["sx"], c["K"]), s["dy"].float()
        if c["E"] == 0:
            return (x.t() @ dy).to(s["dy"].dtype)
        e, there, at = _place(s["offs"], s["tok"].numel())
        xs = _by_expert(x[s["tok"].clamp(min=0).long()], e, there, at, c["E"], s["most"])
        dys = _by_expert(dy, e, there, at, c["E"], s["most"])
        return torch.bmm(xs.transpose(1, 2).contiguous(), dys).to(s["dy"].dtype)
    if c["what"] == "weights":
        return _store_weights(s["w"])
    if c["what"] == "rows":
        q, scale = _store(s["x"])
        return q, scale, _rows(q, scale, c["K"]).to(s["x"].dtype)
    if c["what"] == "gate":
        g, u = s["gate"].float(), s["up"].float()
        return *_store(g / (1 + torch.exp(-g)) * u), *_store(s["gate"]), *_store(s["up"])
    gq, gs, uq, us = s["kept"]
    g, u, dh = _rows(gq, gs, c["K"]), _rows(uq, us, c["K"]), s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    return (dh * u * sig * (1 + g * (1 - sig))).to(s["dh"].dtype), (dh * g * sig).to(s["dh"].dtype)


def _own(s):
    import bit_gemm_token_amd as bgt
    c = s["case"]
    if c["op"] == "balance":
        out = bgt.moe_balance(s["logits"], s["ids"])
        if not c["grad"]:
            return out
        return *out, bgt.moe_balance_backward(s["dloss"], s["logits"], out[1], out[3])
    if c["op"] == "experts":
        q, scale = bgt.quantize_fp8(s["x"])
        y = bgt.w8a8_moe_gemm_fp8(q, scale, s["offs"], s["tok"], s["qw"], s["sw"], out_dtype=s["x"].dtype)
        return q, scale, y
    if c["op"] == "linear":
        y, q, scale = bgt.w8a8_linear_fp8(s["x"], s["qw"], s["sw"])
        return q, scale, y
    if c["op"] == "wgrad":
        if c["E"] == 0:
            return bgt.wgrad_fp8(s["qx"], s["sx"], s["dy"], c["K"])
        return bgt.moe_wgrad_fp8(s["qx"], s["sx"], s["offs"], s["tok"], s["dy"], c["K"])
    if c["what"] == "weights":
        w = bgt.pack_weights_fp8(s["w"], turned=True)
        return w["qw"], w["sw"], w["qt"], w["st"]
    if c["what"] == "rows":
        q, scale = bgt.quantize_fp8(s["x"])
        return q, scale, bgt.dequantize_fp8(q, scale, c["K"], out_dtype=s["x"].dtype)
    if c["what"] == "gate":
        return bgt.silu_mul_fp8(s["gate"], s["up"])
    return bgt.silu_mul_fp8_backward(s["dh"], *s["kept"])


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------- work
def work(case):
    c, b = case, SIZE[case["type"]]
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": b * T * E * (3 if c["grad"] else 1) + 4 * (T * k + 2 * E), "flops": (10 if c["grad"] else 5) * T * E}
    if c["op"] == "store":
        what, K = c["what"], c["K"]
        n = K * (c["N"] if what == "weights" else c["M"])
        stored = 1 + 1 / BLOCK
        return {"weights": {"bytes": n * (b + 2) + 2 * n / BLOCK ** 2, "flops": 2 * n},
                "rows": {"bytes": n * (2 * b + stored), "flops": 3 * n},
                "gate": {"bytes": n * (2 * b + 3 * stored), "flops": 12 * n},
                "gate_grad": {"bytes": n * (3 * b + 2 * stored), "flops": 16 * n}}[what]
    K, N, E = c["K"], c["N"], c.get("E", 0)
    if c["op"] == "linear":
        into, over = (K, N) if c["grad"] else (N, K)
        M = c["M"]
        return {"bytes": K * N + M * (b * (over + into) + over * (1 + 1 / BLOCK)), "flops": 2 * M * K * N}
    if c["op"] == "wgrad" and E == 0:
        return {"bytes": c["M"] * (K * (1 + 1 / BLOCK) + b * N) + b * K * N, "flops": 2 * c["M"] * K * N}
    T, k = (c["M"] if c["op"] == "wgrad" else c["T"]), c["k"]
    R = T * k * (1 - c["pad"])
    if c["op"] == "wgrad":
        return {"bytes": T * K * (1 + 1 / BLOCK) + R * b * N + b * E * K * N + 4 * T * k, "flops": 2 * R * K * N}
    into, over = (K, N) if c["grad"] else (N, K)
    busy = E * (1 - (1 - k / E) ** T)              # experts that some token is sent to
    return {"bytes": busy * K * N + T * over * (b + 1 + 1 / BLOCK) + b * T * k * into + 4 * (E + 1 + T * k),
            "flops": 2 * R * K * N}


# ------------------------------------------------------------------------- exact
def _e4m3(v):
    """v (64 bits) rounded to e4m3, ties to even, saturated: steps of 2^(exponent - 3), no
    finer than 2^-9."""
    _, ex = torch.frexp(v.cpu())
    step = torch.exp2((ex.to(v.device).double() - 4).clamp(min=-9))
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _least(top):
    """The least e with top <= 448 * 2^e by comparison, at least LOW; 2^e in 64 bits."""
    e = torch.floor(torch.log2(top.clamp(min=1e-300) / TOP)) - 1
    e = e + (top > TOP * torch.exp2(e)) + (top > TOP * torch.exp2(e + 1))
    return torch.exp2(e.clamp(min=LOW))


def _exact_store(x):
    """(values, scales as K'/128 x M, what they stand for), in 64 bits."""
    M, K = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -K % BLOCK)).view(M, -1, BLOCK)
    s = _least(v.abs().amax(2))
    q = _e4m3(v / s[..., None])
    return q.view(M, -1), s.t(), (q * s[..., None]).view(M, -1)


def _exact_weights(q, scale):
    """K' x N weights in 64 bits: element (k, n) from value (n, k) and the scale of its block."""
    n = torch.arange(q.shape[0], device=q.device) // BLOCK
    k = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double().t() * scale.double()[k[:, None], n[None, :]]


def _exact_product(x, q, scale):
    """Columns at a time, for the memory."""
    step = 32 * BLOCK
    return torch.cat([x @ _exact_weights(q[j:j + step], scale[:, j // BLOCK:(j + step) // BLOCK])
                      for j in range(0, q.shape[0], step)], 1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "linear":
        q, scale, x = _exact_store(s["x"])
        return q, scale, _exact_product(x, s["qw"], s["sw"])
    if c["op"] in ("experts", "wgrad") and c["E"]:
        offs, tok = s["offs"].tolist(), s["tok"].long()
        spans = [(e, tok[offs[e]:offs[e + 1]], slice(offs[e], offs[e + 1])) for e in range(c["E"])]
    if c["op"] == "experts":
        q, scale, x = _exact_store(s["x"])
        y = torch.zeros(s["tok"].numel(), s["qw"].shape[1], dtype=torch.float64, device=x.device)
        for e, t, at in spans:
            if t.numel():
                y[at] = _exact_product(x[t], s["qw"][e], s["sw"][e])
        return q, scale, y
    if c["op"] == "wgrad":
        k = torch.arange(c["K"], device=s["dy"].device)
        x = s["qx"].double()[:, :c["K"]] * s["sx"].double()[k // BLOCK].t()
        if c["E"] == 0:
            return torch.cat([x[:, j:j + 2048].t() @ s["dy"].double() for j in range(0, c["K"], 2048)])
        return torch.stack([x[t].t() @ s["dy"][at].double() for _, t, at in spans])
    if c["op"] == "store":
        if c["what"] == "weights":
            w = s["w"].double()
            w = torch.nn.functional.pad(w, (0, -w.shape[1] % BLOCK, 0, -w.shape[0] % BLOCK))
            v = w.unfold(0, BLOCK, BLOCK).unfold(1, BLOCK, BLOCK)          # block row, block column, k, n
            scale = _least(v.abs().amax((2, 3)))
            q = _e4m3(v / scale[..., None, None]).permute(0, 2, 1, 3).reshape(w.shape)
            return q[:, :c["N"]].t(), scale, q[:c["K"]], scale.t()
        if c["what"] == "rows":
            q, scale, x = _exact_store(s["x"])
            return q, scale, x[:, :c["K"]]
        if c["what"] == "gate":
            g, u = s["gate"].double(), s["up"].double()
            parts = [_exact_store(v)[:2] for v in (torch.nn.functional.silu(g) * u, g, u)]
            return [t for p in parts for t in p]
        k = torch.arange(c["K"], device=s["dh"].device)
        g, u = (q.double()[:, :c["K"]] * v.double()[k // BLOCK].t() for q, v in (s["kept"][:2], s["kept"][2:]))
        sig, dh = torch.sigmoid(g), s["dh"].double()
        return dh * u * (sig + g * sig * (1 - sig)), dh * g * sig
    v, ids = s["logits"].double().cpu(), s["ids"].cpu()
    E = c["E"]
    there = ~torch.isneginf(v).all(1)
    p = torch.zeros_like(v)
    p[there] = torch.softmax(v[there], 1)
    n = torch.bincount(ids[ids >= 0].long(), minlength=E).double()
    f, tokens = n / max(1.0, float(n.sum())), max(1, int(there.sum()))
    mean = p.sum(0) / tokens
    out = [E * (f @ mean), None, mean, None]
    if c["grad"]:
        out.append(float(s["dloss"].double()) * E / tokens * (p * f - p * (p @ f)[:, None]))
    return out
