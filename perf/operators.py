"""Measured cases of the mixture-of-experts layer's operators around the experts' products.

    route     router logits -> the k experts of each token, their weights, and the tokens
              sorted by expert (offsets, token of each slot, slot of each token); with
              "grad" also the gradient of the logits
    gather    token rows copied to expert order; "grad": rows summed back into the tokens
    combine   expert rows weighted and summed into the tokens; "grad": the rows' and the
              weights' gradients
    gemv      a few rows times one 4-bit weight matrix with a float scale per group of 128
    experts   the same for routed slots, each times its own expert's matrix

`run` computes each operator either in elementary torch operations, in 32 bits and
rounded once at the end, or (`own`) through bit_gemm_token_amd. Sizes are those of the
repository's benchmark (4096, 11008, 14336, 22016; 8 experts, 2 for each token) and
generic ones.
"""
import math

import torch

own = False

GROUP = 128
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # serving, one token: latency of the routing of a decode step
        dict(name="route_one", op="route", T=1, E=8, k=2, type="f32", norm="chosen", pad=0.0, grad=False),
        # a prompt of 4096 tokens, some of them padding that no expert takes; bf16 logits tie often
        dict(name="route_prompt", op="route", T=4096, E=8, k=2, type="bf16", norm="chosen", pad=0.05, grad=False),
        # a training batch (odd count) over many small experts, with the router's gradient
        dict(name="route_train", op="route", T=16381, E=64, k=6, type="f32", norm="all", pad=0.0, grad=True),
        # the same prompt's rows copied to expert order
        dict(name="gather_prompt", op="gather", T=4096, H=4096, E=8, k=2, type="bf16", pad=0.0, grad=False),
        # gradient of that copy at odd sizes, in fp32, with padding tokens
        dict(name="gather_grad", op="gather", T=1021, H=1000, E=60, k=4, type="f32", pad=0.1, grad=True),
        # a decode batch of 16: expert rows back to the tokens
        dict(name="combine_decode", op="combine", T=16, H=4096, E=8, k=2, type="bf16", pad=0.0, grad=False),
        # a training batch: gradients of expert rows and of the router's weights
        dict(name="combine_train", op="combine", T=4096, H=4096, E=8, k=2, type="bf16", pad=0.0, grad=True),
        # one token times an attention projection: latency
        dict(name="gemv_one", op="gemv", M=1, K=4096, N=4096, type="bf16"),
        # a decode batch times the widest layer of the benchmark
        dict(name="gemv_batch", op="gemv", M=16, K=4096, N=22016, type="f16"),
        # a few fp32 rows times a down projection with an odd group count
        dict(name="gemv_down", op="gemv", M=3, K=11008, N=4096, type="f32"),
        # one token through two of eight experts' up projections
        dict(name="experts_one", op="experts", T=1, E=8, k=2, K=4096, N=14336, type="bf16", pad=0.0),
        # a decode batch (odd count) through all experts' down projections
        dict(name="experts_batch", op="experts", T=61, E=8, k=2, K=14336, N=4096, type="f16", pad=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gather", "combine", "gemv", "experts"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "route":
        E = _log(rng, 4, 256)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)), type=kind,
                    norm=rng.choice(["chosen", "all"]), pad=rng.choice([0.0, 0.05, 0.3]),
                    grad=rng.random() < 0.5)
    if op in ("gather", "combine"):
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:                      # hidden sizes are mostly multiples of 64
            H = max(64, H // 64 * 64)
        T = min(_log(rng, 1, 8192), max(1, (1 << 25) // (k * H)))
        return dict(op=op, T=T, H=H, E=E, k=k, type=kind, pad=rng.choice([0.0, 0.1]),
                    grad=rng.random() < 0.5)
    K, N = GROUP * _log(rng, 2, 112), 16 * _log(rng, 4, 1376)
    if op == "gemv":
        return dict(op=op, M=_log(rng, 1, 64), K=K, N=N, type=kind)
    E = _log(rng, 4, 64)
    most = 8 * 4096 * 14336 // (E * K)
    N = max(64, min(N, most // 16 * 16))
    return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), K=K, N=N, type=kind,
                pad=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------------ inputs
def _logits(g, T, E, pad, dev):
    """Normal logits with a bias per expert, as trained routers give; of a padding
    token every logit is -inf, and a few other entries are masked too."""
    logits = torch.randn(T, E, generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
    if pad:
        gone = torch.rand(T, 1, generator=g, device=dev) < pad
        some = torch.rand(T, E, generator=g, device=dev) < 0.1 * pad
        logits = logits.masked_fill(gone | some, -math.inf)
    return logits


def _activations(g, T, K, dev):
    """Normal rows with one channel in a hundred twenty times as large."""
    x = torch.randn(T, K, generator=g, device=dev)
    x[:, torch.randperm(K, generator=g, device=dev)[: max(1, K // 100)]] *= 20
    return x


def _pack(g, K, N, dev):
    """A normal weight matrix (some salient elements) in 4 bits: the library's packed
    layout and the scales of the groups."""
    w = 0.02 * torch.randn(K, N, generator=g, device=dev)
    w[torch.rand(K, N, generator=g, device=dev) < 0.001] *= 10
    w = w.view(K // GROUP, GROUP, N)
    s = w.abs().amax(1) / 7
    q = torch.round(w / s[:, None]).clamp_(-7, 7).to(torch.int32)
    q = q.view(K // GROUP, 2, 4, 2, 2, 4, N // 16, 16).permute(6, 0, 2, 7, 1, 3, 5, 4) & 15
    return (q[..., 0] | q[..., 1] << 4).to(torch.uint8).reshape(-1), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, dt = case, TYPES[case["type"]]
    s = {"case": dict(case)}
    if c["op"] == "gemv":
        s["x"] = _activations(g, c["M"], c["K"], dev).to(dt)
        s["packed"], s["fscale"] = _pack(g, c["K"], c["N"], dev)
        return s
    logits = _logits(g, c["T"], c["E"], c["pad"], dev)
    if c["op"] == "route":
        s["logits"] = logits.to(dt)
        if c["grad"]:
            s["dweights"] = torch.randn(c["T"], c["k"], generator=g, device=dev)
        return s
    # the routing that such a program already holds
    s["weights"], ids = _top(logits, c["k"], "chosen")
    s["ids"] = ids
    s["offs"], s["tok"], s["pos"] = _sort(ids, c["E"])
    R = c["T"] * c["k"]
    if c["op"] == "experts":
        s["x"] = _activations(g, c["T"], c["K"], dev).to(dt)
        both = [_pack(g, c["K"], c["N"], dev) for _ in range(c["E"])]
        s["packed"] = torch.stack([p for p, _ in both])
        s["fscale"] = torch.stack([f for _, f in both])
    elif c["op"] == "gather":
        rows = R if c["grad"] else c["T"]
        s["rows"] = torch.randn(rows, c["H"], generator=g, device=dev).to(dt)
    else:
        s["ys"] = torch.randn(R, c["H"], generator=g, device=dev).to(dt)
        if c["grad"]:
            s["dy"] = torch.randn(c["T"], c["H"], generator=g, device=dev).to(dt)
    return s


# ------------------------------------------------------------------- plain forms
def _top(logits, k, norm):
    """The k largest logits of each row, ties to the lower expert; an expert at -inf is
    not taken (id -1, weight 0)."""
    v = logits.float()
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    gone = top == -math.inf
    m = top[:, :1].masked_fill(gone[:, :1], 0.0)
    e = torch.exp(top - m)
    total = e.sum(1, keepdim=True) if norm == "chosen" else torch.exp(v - m).sum(1, keepdim=True)
    w = torch.where(gone, 0.0, e / torch.where(total > 0, total, 1.0))
    return w, ids.masked_fill(gone, -1).to(torch.int32)


def _sort(ids, E):
    """Slots sorted by expert, tokens in order within an expert."""
    T, k = ids.shape
    key = torch.where(ids < 0, E, ids.long()).view(-1)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offs = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    gone = key[order] == E
    tok = (order // k).masked_fill(gone, -1).to(torch.int32)
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=ids.device))
    return offs, tok, pos.masked_fill(key == E, -1).view(T, k).to(torch.int32)


def _route_grad(dw, logits, ids, norm):
    """Gradient of the logits: w_i (dw_i - sum_j w_j dw_j), over the chosen experts or all."""
    v = logits.float()
    chosen = ids >= 0
    at = ids.clamp(min=0).long()
    top = v.gather(1, at).masked_fill(~chosen, -math.inf)
    base = top if norm == "chosen" else v
    m = base.amax(1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    e = torch.exp(base - m)
    p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    dw = dw.masked_fill(~chosen, 0.0)
    if norm == "chosen":
        d = p * (dw - (p * dw).sum(1, keepdim=True))
        return torch.zeros_like(v).scatter_add_(1, at, d.masked_fill(~chosen, 0.0)).to(logits.dtype)
    full = torch.zeros_like(v).scatter_add_(1, at, dw)
    return (p * (full - (p * full).sum(1, keepdim=True))).to(logits.dtype)


def _rows_of(rows, pos):
    """rows[pos] with zeros where a token has no slot: T x k x H."""
    got = rows[pos.clamp(min=0).long()].float()
    return torch.where(pos[..., None] >= 0, got, 0.0)


def _unpack(packed, fscale):
    """The weights that the packed codes and scales stand for: (..., K, N) in fp32."""
    G, N = fscale.shape[-2:]
    lead = fscale.shape[:-2]
    b = packed.view(-1, N // 16, G, 4, 16, 2, 2, 4)
    q = torch.stack([b & 15, b >> 4], -1).permute(0, 2, 5, 3, 6, 8, 7, 1, 4).reshape(-1, G, GROUP, N)
    q = ((q ^ 8).to(torch.int8) - 8).float()
    return (q * fscale.view(-1, G, 1, N)).view(*lead, G * GROUP, N)


def _expert_of(offs, R):
    """Expert of each slot (the number of offsets at or below it, less one)."""
    r = torch.arange(R, device=offs.device)
    return (r[:, None] >= offs[None, 1:]).sum(1), r


def _experts(x, offs, tok, packed, fscale):
    """y[r] = x[tok[r]] times the matrix of the expert of slot r; zero past the last slot."""
    (E, G, N), (T, K), R = fscale.shape, x.shape, tok.numel()
    e, r = _expert_of(offs, R)
    there = (e < E)[:, None]
    e = e.clamp(max=E - 1)
    rows = torch.where(there, x.float()[tok.clamp(min=0).long()], 0.0)
    if R <= E:                                    # fewer slots than experts: a matrix for each slot
        y = torch.bmm(rows[:, None], _unpack(packed[e], fscale[e]))[:, 0]
    else:                                         # an expert has at most T slots
        at = (r - offs[e]).clamp(max=T - 1)
        full = rows.new_zeros(E, T, K).index_put_((e, at), rows, accumulate=True)
        y = torch.bmm(full, _unpack(packed, fscale))[e, at]
    return torch.where(there, y, 0.0).to(x.dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "gemv":
        return (s["x"].float() @ _unpack(s["packed"], s["fscale"])).to(s["x"].dtype)
    if c["op"] == "experts":
        return _experts(s["x"], s["offs"], s["tok"], s["packed"], s["fscale"])
    if c["op"] == "route":
        w, ids = _top(s["logits"], c["k"], c["norm"])
        out = (w, ids, *_sort(ids, c["E"]))
        return out + (_route_grad(s["dweights"], s["logits"], ids, c["norm"]),) if c["grad"] else out
    if c["op"] == "gather":
        if c["grad"]:
            return _rows_of(s["rows"], s["pos"]).sum(1).to(s["rows"].dtype)
        xs = s["rows"][s["tok"].clamp(min=0).long()]
        return torch.where(s["tok"][:, None] >= 0, xs, 0.0)
    ys = _rows_of(s["ys"], s["pos"])
    if not c["grad"]:
        return (s["weights"][..., None] * ys).sum(1).to(s["ys"].dtype)
    dy = s["dy"].float()
    w = torch.zeros(s["tok"].numel(), device=dy.device)
    w[s["pos"][s["pos"] >= 0].long()] = s["weights"][s["pos"] >= 0]
    dys = (w[:, None] * dy[s["tok"].clamp(min=0).long()]).to(s["ys"].dtype)
    return dys, (ys * dy[:, None]).sum(2)


def _own(s):
    import bit_gemm_token_amd as bgt
    c = s["case"]
    if c["op"] == "gemv":
        return bgt.w4a16_gemv(s["x"], s["packed"], s["fscale"], c["N"])
    if c["op"] == "experts":
        return bgt.w4a16_moe_gemv(s["x"], s["offs"], s["tok"], s["packed"], s["fscale"], c["N"])
    if c["op"] == "route":
        out = bgt.moe_route(s["logits"], c["k"], norm=c["norm"])
        if not c["grad"]:
            return out
        return *out, bgt.moe_route_backward(s["dweights"], s["logits"], out[1], norm=c["norm"])
    if c["op"] == "gather":
        if c["grad"]:
            return bgt.moe_gather_backward(s["rows"], s["pos"])
        return bgt.moe_gather(s["rows"], s["offs"], s["pos"])
    if c["grad"]:
        return bgt.moe_combine_backward(s["dy"], s["ys"], s["offs"], s["pos"], s["weights"])
    return bgt.moe_combine(s["ys"], s["pos"], s["weights"])


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------- work
def work(case):
    c, b = case, SIZE[case["type"]]
    if c["op"] == "gemv":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": K * N / 2 + 4 * (K // GROUP) * N + b * M * (K + N), "flops": 2 * M * K * N}
    T, E, k = c["T"], c["E"], c["k"]
    R = T * k
    if c["op"] == "experts":
        K, N = c["K"], c["N"]
        busy = E * (1 - (1 - k / E) ** T)          # experts that some token is sent to
        return {"bytes": busy * (K * N / 2 + 4 * (K // GROUP) * N) + b * (T * K + R * N) + 4 * (E + 1 + R),
                "flops": 2 * R * K * N}
    if c["op"] == "route":
        one = b * T * E + 4 * (4 * R + E + 1)
        return {"bytes": one + (b * T * E + 4 * R if c["grad"] else 0), "flops": 5 * T * E}
    H = c["H"]
    if c["op"] == "gather":
        return {"bytes": b * H * (T + R) + 4 * R, "flops": R * H if c["grad"] else 0}
    if c["grad"]:
        return {"bytes": b * H * (T + 2 * R) + 12 * R, "flops": 3 * R * H}
    return {"bytes": b * H * (T + R) + 8 * R, "flops": 2 * R * H}


# ------------------------------------------------------------------------- exact
def _exact_weights(packed, fscale, K, N):
    """W[k][j] in 64 bits from the layout's index formula (one matrix): columns of 16,
    groups of 128, 16 bytes for each of 64 lanes, low nibbles first."""
    k = torch.arange(K, device=packed.device)[:, None]
    j = torch.arange(N, device=packed.device)[None, :]
    r, e = k % GROUP, k % 16
    lane = 16 * ((r % 64) // 16) + j % 16
    byte = (((j // 16) * (K // GROUP) + k // GROUP) * 64 + lane) * 16 + 8 * (r // 64) + 4 * (e // 8) + e % 4
    code = (packed[byte].int() >> (4 * ((e % 8) // 4))) & 15
    code = torch.where(code > 7, code - 16, code)
    return code.double() * fscale.double().repeat_interleave(GROUP, 0)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "gemv":
        parts = []
        for j in range(0, c["N"], 2048):           # columns at a time, for the memory
            n = min(2048, c["N"] - j)
            half = s["packed"][j * c["K"] // 2: (j + n) * c["K"] // 2]
            parts.append(s["x"].double() @ _exact_weights(half, s["fscale"][:, j:j + n], c["K"], n))
        return torch.cat(parts, 1)
    if c["op"] == "experts":
        y = torch.zeros(s["tok"].numel(), c["N"], dtype=torch.float64, device=s["x"].device)
        offs = s["offs"].tolist()
        for e in range(c["E"]):
            if offs[e] < offs[e + 1]:
                rows = s["x"][s["tok"][offs[e]:offs[e + 1]].long()].double()
                for j in range(0, c["N"], 2048):
                    n = min(2048, c["N"] - j)
                    half = s["packed"][e][j * c["K"] // 2: (j + n) * c["K"] // 2]
                    y[offs[e]:offs[e + 1], j:j + n] = rows @ _exact_weights(half, s["fscale"][e][:, j:j + n], c["K"], n)
        return y
    if c["op"] == "route":
        v = s["logits"].double().cpu()
        # the rank of an entry: larger ones, and equal ones before it
        T, E = v.shape
        ids = torch.full((T, c["k"]), -1)
        earlier = torch.ones(E, E).tril(-1).bool()          # [i, j]: j before i
        for t in range(0, T, 512):
            u = v[t:t + 512]
            rank = ((u[:, None, :] > u[:, :, None]) | ((u[:, None, :] == u[:, :, None]) & earlier)).sum(2)
            row, i = torch.nonzero((rank < c["k"]) & (u > -math.inf), as_tuple=True)
            ids[t + row, rank[row, i]] = i
        chosen = ids >= 0
        mask = torch.zeros(T, E + 1, dtype=torch.bool).scatter_(1, torch.where(chosen, ids, E), True)[:, :E]
        kept = v if c["norm"] == "all" else v.masked_fill(~mask, -math.inf)
        p = torch.softmax(kept, 1).nan_to_num(0.0)          # a row with nothing left: zeros
        w = torch.where(chosen, p.gather(1, ids.clamp(min=0)), 0.0)
        out = [w, None, None, None, None]
        if c["grad"]:
            dp = torch.zeros(T, E + 1, dtype=torch.float64)
            dp.scatter_(1, torch.where(chosen, ids, E), s["dweights"].double().cpu())
            dp = dp[:, :E]
            out.append(p * dp - p * (p * dp).sum(1, keepdim=True))
        return out
    pos, there = s["pos"].cpu().long(), s["pos"].cpu() >= 0
    T, k = pos.shape
    if c["op"] == "gather":
        rows = s["rows"].double().cpu()
        if c["grad"]:
            out = torch.zeros(T, c["H"], dtype=torch.float64)
            for j in range(k):
                out[there[:, j]] += rows[pos[there[:, j], j]]
            return out
        out = torch.zeros(T * k, c["H"], dtype=torch.float64)
        for j in range(k):
            out[pos[there[:, j], j]] = rows[there[:, j]]
        return out
    ys, w = s["ys"].double().cpu(), s["weights"].double().cpu()
    if not c["grad"]:
        out = torch.zeros(T, c["H"], dtype=torch.float64)
        for j in range(k):
            m = there[:, j]
            out[m] += w[m, j, None] * ys[pos[m, j]]
        return out
    dy = s["dy"].double().cpu()
    dys, dw = torch.zeros_like(ys), torch.zeros(T, k, dtype=torch.float64)
    for j in range(k):
        m = there[:, j]
        dys[pos[m, j]] = w[m, j, None] * dy[m]
        dw[m, j] = (ys[pos[m, j]] * dy[m]).sum(1)
    return dys, dw
