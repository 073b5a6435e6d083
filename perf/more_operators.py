"""What the expert selection and the low-rank adapters are measured on.

Two operators, each forward alone and as a training step, in several sizes:

  select     router logits to the experts of each token and their weights; as a training step also d_logits
  adapters   base + scale (x A^T) B^T with one pair (A, B) per request; as a training step also x A^T, dx, dA, dB

``own`` False computes them with elementary torch operations, ``own`` True
through the library.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def _select(M, E, top_k, dtype, score="softmax", bias=False, groups=1, top_groups=1, group_picks=1, renormalise=True,
            scale=1.0, off=0.0, train=False, name=None):
    c = {"op": "select", "M": M, "E": E, "top_k": top_k, "dtype": dtype, "score": score, "bias": bias,
         "groups": groups, "top_groups": top_groups, "group_picks": group_picks, "renormalise": renormalise,
         "scale": scale, "off": off, "train": train}
    return c if name is None else {"name": name, **c}


def _adapters(M, K, N, L, r, dtype, runs, none=0.0, order=True, train=False, name=None):
    """runs: the tokens of a request lie together, as prompts do; else each token is of any request. none: the
    share of tokens without an adapter. order: the program keeps the tokens sorted by adapter."""
    c = {"op": "adapters", "M": M, "K": K, "N": N, "L": L, "r": r, "dtype": dtype, "runs": runs, "none": none,
         "order": order, "train": train}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # the MoE block's decode step: launch latency
        _select(32, 256, 8, "f32", name="select 32 tokens"),
        # a prompt of odd length, balanced by a bias, experts limited to groups
        _select(4099, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, name="select in groups 4099 tokens"),
        # a training batch of a small MoE with plain softmax weights: the gradient reaches every expert
        _select(16384, 60, 4, "f16", renormalise=False, train=True, name="select plain 16384 tokens"),
        # a long training batch, balanced by a bias, some experts switched off
        _select(131072, 256, 8, "bf16", "sigmoid", True, off=0.02, train=True, name="select with bias 131072 tokens"),
        # decode, one token
        _adapters(1, 4096, 4096, 8, 16, "f16", False, order=False, name="adapters 1 token"),
        # decode, a batch of many requests on the widest matrix of the dense stack
        _adapters(64, 4096, 28672, 64, 16, "bf16", False, 0.1, name="adapters 64 requests"),
        # prompts of a few requests on the FFN pair's first matrix, an order for this call only
        _adapters(1777, 5120, 17408, 16, 64, "f16", True, 0.1, order=False, name="adapters 1777 tokens"),
        # long prompts of many requests on the way down
        _adapters(8192, 14336, 4096, 32, 8, "bf16", True, 0.05, name="adapters 8192 tokens"),
        # a small step of odd sizes
        _adapters(257, 2048, 2047, 3, 5, "f16", True, 0.2, train=True, name="train 257 tokens"),
        # one step for many adapters, tokens in any order
        _adapters(4000, 2048, 2048, 96, 32, "f16", False, train=True, name="train 96 adapters"),
        # fine-tuning one adapter
        _adapters(8192, 4096, 14336, 1, 16, "bf16", True, train=True, name="train 8192 tokens"),
        # fine-tuning several wide ones together
        _adapters(8192, 4096, 14336, 8, 64, "bf16", True, train=True, name="train 8 wide adapters"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    train = rng.random() < 0.5
    if rng.random() < 0.45:
        score, bias = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
        if rng.random() < 0.4:
            groups, each = rng.randint(2, 16), _log(rng, 2, 64)
            E, top_groups = groups * each, rng.randint(1, groups)
            picks = rng.randint(1, 2)
        else:
            E, groups, top_groups, picks, each = _log(rng, 2, 1024), 1, 1, 1, 0
        top_k = rng.randint(1, min(16, top_groups * each if groups > 1 else E))
        M = _log(rng, 1, min(131072, (1 << 25) // E))
        return _select(M, E, top_k, rng.choice(["f32", "bf16", "f16"]), score, bias, groups, top_groups, picks,
                       top_k > 1 and rng.random() < 0.7, rng.choice([1.0, 2.5]),
                       rng.choice([0.0, 0.05]) if E >= 16 else 0.0, train)
    K, N = 128 * _log(rng, 1, 112), _log(rng, 8, 28672)
    L, r = _log(rng, 1, 256), _log(rng, 1, 128)
    # the plain form multiplies every token by every adapter
    most = min((1 << 27) // (K + N), 77_000_000_000 // (L * r * (K + N)), (1 << 32) // (4 * L * r))
    M = _log(rng, 1, max(1, min(16384, most)))
    return _adapters(M, K, N, L, r, rng.choice(["f16", "bf16"]), rng.random() < 0.6, rng.choice([0.0, 0.1, 0.5]),
                     rng.random() < 0.7, train)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, dtype, g):
    """Normal values; one channel in about 64 is twenty times the rest, as in a transformer's residual stream."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x *= torch.where(torch.rand(cols, device="cuda", generator=g) < 1 / 64, 20.0, 1.0)
    return x.to(DT[dtype])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    M = case["M"]
    if case["op"] == "select":
        E, k = case["E"], case["top_k"]
        # some experts are preferred
        logits = torch.randn(M, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
        logits[:, torch.rand(E, device="cuda", generator=g) < case["off"]] = -math.inf
        s["logits"] = logits.to(DT[case["dtype"]])
        s["b"] = None
        if case["bias"]:   # moved by steps of a thousandth
            s["b"] = (0.05 * torch.randn(E, device="cuda", generator=g) * 1000).round() / 1000
        if case["train"]:
            s["dw"] = 0.01 * torch.randn(M, k, device="cuda", generator=g)
        return s
    K, N, L, r, dt = case["K"], case["N"], case["L"], case["r"], DT[case["dtype"]]
    s["x"] = _activations(M, K, case["dtype"], g)
    s["A"] = (torch.randn(L, r, K, device="cuda", generator=g) / math.sqrt(K)).to(dt)
    s["B"] = (0.02 * torch.randn(L, N, r, device="cuda", generator=g)).to(dt)
    s["scales"] = 2.0 ** torch.randint(-1, 3, (L,), device="cuda", generator=g).float()
    s["base"] = torch.randn(M, N, device="cuda", generator=g).to(dt)      # what the shared projection gave
    if case["runs"]:
        # requests of about equal length, in any order of their adapters
        n = max(L, 4)
        of = torch.randint(0, L, (n,), device="cuda", generator=g)
        of[torch.rand(n, device="cuda", generator=g) < case["none"]] = -1
        ids = of[torch.arange(M, device="cuda") * n // M]
    else:
        ids = torch.randint(0, L, (M,), device="cuda", generator=g)
        ids[torch.rand(M, device="cuda", generator=g) < case["none"]] = -1
    s["ids"] = ids.to(torch.int32)
    s["sorted"] = None
    if case["order"]:
        kept = torch.where(ids >= 0, ids, L)
        perm = torch.sort(kept, stable=True).indices
        counts = torch.bincount(kept, minlength=L + 1)[:L]
        perm[int(counts.sum()):] = -1
        s["sorted"] = (torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), perm.to(torch.int32))
    if case["train"]:
        # gradients as a loss scaled for 16 bits gives them
        s["dy"] = (0.01 * torch.randn(M, N, device="cuda", generator=g)).to(dt)
        s["dbase"] = (0.01 * torch.randn(M, K, device="cuda", generator=g)).to(dt)   # the shared projection's dx
    return s


# ---------------------------------------------------------------- plain form

def _plain_select(s):
    """The order of experts is decided in 64 bits: values next to each other are common among many tokens."""
    M, E, k = s["M"], s["E"], s["top_k"]
    G, each = s["groups"], s["E"] // s["groups"]
    wide = s["logits"].double()
    if s["score"] == "softmax":
        e = torch.exp(wide - wide.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-wide))
    there = wide > -math.inf
    # without a bias experts go by their logits: the scores rise with them
    c = p if s["b"] is not None or G > 1 else wide
    if s["b"] is not None:
        c = c + s["b"].double()
    c = torch.where(there, c, -math.inf)
    if G > 1:
        best = torch.sort(c.reshape(M, G, each), dim=2, descending=True).values[..., :s["group_picks"]]
        value = torch.where(best > -math.inf, best, 0).sum(2)
        value = torch.where(best[..., 0] > -math.inf, value, -math.inf)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        kept = torch.zeros(M, G, dtype=torch.bool, device=c.device)
        kept[torch.arange(M, device=c.device)[:, None], order[:, :s["top_groups"]]] = True
        c = torch.where(kept[..., None].expand(M, G, each).reshape(M, E), c, -math.inf)
    top = torch.sort(c, dim=1, descending=True, stable=True)
    ids = torch.where(top.values[:, :k] > -math.inf, top.indices[:, :k], -1)
    picked = ids >= 0
    at = ids.clamp(min=0)
    rows = torch.arange(M, device=c.device)[:, None]
    w = torch.where(picked, p[rows, at], 0).float()
    total = w.sum(1, keepdim=True)
    if s["renormalise"]:
        w = torch.where(total > 0, w / total, 0)
    out = {"ids": ids.to(torch.int32), "weights": s["scale"] * w}
    if s["train"]:
        pf = torch.where(there, p, 0).float()
        g = torch.where(picked, s["scale"] * s["dw"], 0)
        if s["renormalise"]:
            g = torch.where(picked & (total > 0), (g - (w * g).sum(1, keepdim=True)) / total, 0)
        # an id of -1 stands at 0 and adds nothing there
        ds = torch.zeros(M, E, device=c.device).scatter_add_(1, at, g * picked)
        if s["score"] == "softmax":
            d = pf * (ds - (pf * ds).sum(1, keepdim=True))
        else:
            d = ds * pf * torch.where(there, 1 / (1 + torch.exp(wide)), 0).float()
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_adapters(s):
    M, K, N, L, r = s["M"], s["K"], s["N"], s["L"], s["r"]
    dt = s["x"].dtype
    x, ids = s["x"].float(), s["ids"].long()
    a = s["A"].float().reshape(L * r, K)
    b = s["B"].float().permute(0, 2, 1).reshape(L * r, N)
    mine = (torch.arange(L, device="cuda") == ids[:, None])[..., None]        # [M][L][1]
    scale = s["scales"].reshape(1, L, 1)
    every = torch.where(mine, (x @ a.t()).reshape(M, L, r), 0)
    out = {"y": (s["base"].float() + (every * scale).reshape(M, L * r) @ b).to(dt)}
    if s["train"]:
        dy = s["dy"].float()
        out["h"] = every.sum(1)
        u = torch.where(mine, scale * (dy @ b.t()).reshape(M, L, r), 0).reshape(M, L * r)
        out["dx"] = (s["dbase"].float() + u @ a).to(dt)
        out["dA"] = (u.t() @ x).reshape(L, r, K)
        out["dB"] = ((every * scale).reshape(M, L * r).t() @ dy).reshape(L, r, N).permute(0, 2, 1).contiguous()
    return out


# ---------------------------------------------------------------- the library

def _own(s):
    from bit_weight_only_amd import lbq

    if s["op"] == "select":
        how = {"score": lbq.SCORE_SIGMOID if s["score"] == "sigmoid" else lbq.SCORE_SOFTMAX, "groups": s["groups"],
               "top_groups": s["top_groups"], "group_picks": s["group_picks"], "renormalise": s["renormalise"],
               "scale": s["scale"]}
        ids, weights = lbq.moe_select(s["logits"], s["top_k"], bias=s["b"], **how)
        out = {"ids": ids, "weights": weights}
        if s["train"]:
            out["d_logits"] = lbq.moe_select_backward(s["dw"], s["logits"], ids, score=how["score"],
                                                      renormalise=s["renormalise"], scale=s["scale"])
        return out
    ad = lbq.Adapters(s["A"], s["B"], s["scales"])
    if not s["train"]:
        return {"y": lbq.adapters_forward(ad, s["x"], s["ids"], base=s["base"], order=s["sorted"])}
    h = torch.empty(s["M"], s["r"], device="cuda")
    y = lbq.adapters_forward(ad, s["x"], s["ids"], base=s["base"], order=s["sorted"], h=h)
    dx, dA, dB = lbq.adapters_backward(ad, s["dy"], s["x"], h, s["ids"], base=s["dbase"], order=s["sorted"])
    return {"y": y, "h": h, "dx": dx, "dA": dA, "dB": dB}


def run(state):
    if own:
        return _own(state)
    return _plain_select(state) if state["op"] == "select" else _plain_adapters(state)


# ---------------------------------------------------------------- floors and 64 bits

def work(case):
    M = case["M"]
    z = SIZE[case["dtype"]]
    if case["op"] == "select":
        E, k = case["E"], case["top_k"]
        nbytes, flops = M * E * z + 8 * M * k + (4 * E if case["bias"] else 0), 4 * M * E
        if case["train"]:
            nbytes, flops = nbytes + M * E * z + 4 * M * k, 2 * flops
        return {"bytes": nbytes, "flops": flops}
    K, N, L, r = case["K"], case["N"], case["L"], case["r"]
    kept = M * (1 - case["none"])
    drawn = min(kept, max(L, 4)) if case["runs"] else kept
    seen = L * (1 - (1 - 1 / L) ** drawn)                      # adapters that get a token
    # base and y of every token; x, h only where there is an adapter
    nbytes, flops = 2 * M * N * z + kept * K * z + seen * r * (K + N) * z + 4 * M, 2 * kept * r * (K + N)
    if case["train"]:
        nbytes += kept * N * z + 2 * M * K * z + 4 * M * r + 4 * L * r * (K + N)   # dy; dx and its base; h; dA, dB
        flops *= 3
    return {"bytes": int(nbytes), "flops": int(flops)}


def _exact_select(s):
    M, k = s["M"], s["top_k"]
    l = s["logits"].double()
    off = torch.isinf(l)
    l = torch.where(off, -1e5, l).requires_grad_()      # exp of it is nothing in 64 bits
    p = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
    with torch.no_grad():
        c = p + (0 if s["b"] is None else s["b"].double())
        c[off] = -math.inf
        if s["groups"] > 1:
            part = c.reshape(M, s["groups"], -1)
            first = part.amax(2)
            value = first
            if s["group_picks"] == 2:
                rest = part.scatter(2, part.argmax(2, keepdim=True), -math.inf).amax(2)
                value = first + torch.where(torch.isinf(rest), 0.0, rest)
            order = value.argsort(dim=1, descending=True, stable=True)
            lost = torch.zeros_like(value, dtype=torch.bool).scatter(1, order[:, s["top_groups"]:], True)
            c = torch.where(lost[..., None], -math.inf, part).reshape(M, -1)
        picks = c.argsort(dim=1, descending=True, stable=True)[:, :k]
        live = ~torch.isinf(c.gather(1, picks))
    w = p.gather(1, picks) * live
    if s["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = s["scale"] * w
    out = {"ids": None, "weights": w.detach()}
    if s["train"]:
        d = torch.autograd.grad(w, l, s["dw"].double())[0]
        out["d_logits"] = torch.where(d.abs() < 1e-14, 0.0, d)     # a lone expert's is zero but for rounding
    return out


def _exact_adapters(s):
    x, base = s["x"].double(), s["base"].double()
    out = {"y": base}
    if s["train"]:
        out["h"] = x.new_zeros(s["M"], s["r"])
        out["dx"] = s["dbase"].double()
        out["dA"], out["dB"] = torch.zeros_like(s["A"], dtype=torch.double), torch.zeros_like(s["B"], dtype=torch.double)
    for i in sorted(set(s["ids"].tolist()) - {-1}):
        t = (s["ids"] == i).nonzero()[:, 0]
        a, b, scale = s["A"][i].double(), s["B"][i].double(), float(s["scales"][i])
        h = x[t] @ a.t()
        out["y"][t] += scale * (h @ b.t())
        if s["train"]:
            dy = s["dy"][t].double()
            u = scale * (dy @ b)
            out["h"][t] = h
            out["dx"][t] += u @ a
            out["dA"][i] = u.t() @ x[t]
            out["dB"][i] = scale * (dy.t() @ h)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_select(s) if case["op"] == "select" else _exact_adapters(s)
