"""Cases of the sparse SwiGLU layer: routing, grouped expert products, and the
norms with gate and residual around the layer.

For each case ``run`` computes one operator, either in a plain form
(elementary torch operations in 32 bits, rounded once at the end) or through
the library's own entry point.  ``exact`` gives the same outputs from the
definitions in 64 bits.

    route   top-k of the router's logits, softmax weights, and the expert order
    up      Y[p] = SiLU(A[rows[p]] W1[e]) * (A[rows[p]] W2[e]),  p in expert e's range
    down    Z[p] = X[p] W[e]
    norm    z = sum_j w[t,j] Z[slot[t,j]] (or Z[t]);
            R' = s R + g * RMSNorm(z; gamma_post);  H = RMSNorm(R'; gamma_pre)
"""
import math

import torch

own = False

EPS = 1e-6


# ---- cases -----------------------------------------------------------------


def listed():
    return [
        # one token of a serving loop: 8 of 64 experts; pure latency
        {"name": "route-token", "op": "route", "T": 1, "E": 64, "k": 8, "fp32": False, "renorm": True, "pad": 0.0},
        # a long prompt batch, some of its rows padding (every logit -inf)
        {"name": "route-prompt", "op": "route", "T": 16384, "E": 64, "k": 8, "fp32": True, "renorm": False, "pad": 0.03},
        # one token through fine-grained experts: a stream of 8 experts' weights
        {"name": "up-token", "op": "up", "T": 1, "E": 64, "k": 8, "K": 2048, "N": 1024},
        # a decode batch of odd size: nearly every expert gets a few rows
        {"name": "up-batch", "op": "up", "T": 61, "E": 64, "k": 8, "K": 2048, "N": 1024},
        # a short prompt through 8 experts of the 0.5B projection's shape
        {"name": "up-0.5b-prompt", "op": "up", "T": 509, "E": 8, "k": 2, "K": 896, "N": 4864},
        # a long prompt through fine-grained experts, about 1000 rows each
        {"name": "up-prompt", "op": "up", "T": 8192, "E": 64, "k": 8, "K": 2048, "N": 1024},
        # a long prompt through 8 experts of the 7B projection's shape
        {"name": "up-7b-prompt", "op": "up", "T": 4099, "E": 8, "k": 2, "K": 3584, "N": 18944},
        # the down products of the same layers
        {"name": "down-token", "op": "down", "T": 1, "E": 64, "k": 8, "K": 1024, "N": 2048},
        {"name": "down-prompt", "op": "down", "T": 8192, "E": 64, "k": 8, "K": 1024, "N": 2048},
        # the layer's end for one token: 8 experts' rows joined, both norms
        {"name": "norm-token", "op": "norm", "T": 1, "D": 2048, "k": 8, "fp32": False, "gate": "vector"},
        # the same for a long prompt
        {"name": "norm-prompt", "op": "norm", "T": 8192, "D": 2048, "k": 8, "fp32": False, "gate": "vector"},
        # a dense block's end at the 72B width: 32-bit residual stream, a gate of its own for every row
        {"name": "norm-dense", "op": "norm", "T": 8191, "D": 8192, "k": 0, "fp32": True, "gate": "rows"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "up", "up", "down", "down", "norm"])
    if op == "route":
        E = rng.choice([4, 8, 16, 60, 64, 128, 256])
        return {"op": op, "T": _log(rng, 1, 32768), "E": E, "k": rng.randint(1, min(8, E)), "fp32": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "pad": rng.choice([0.0, 0.1])}
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "D": 8 * _log(rng, 64, 1024), "k": rng.choice([0, 0, 1, 2, 4, 8]),
                "fp32": rng.random() < 0.5, "gate": rng.choice(["none", "vector", "rows"])}
    while True:
        E = rng.choice([4, 8, 16, 32, 64])
        c = {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E)), "K": 8 * _log(rng, 64, 512), "N": 8 * _log(rng, 64, 1024)}
        if 3072 not in (c["T"], c["K"], c["N"]) and c["E"] * c["K"] * c["N"] < 3e8 and c["T"] * c["k"] * c["K"] * c["N"] < 3e11 and c["T"] * c["k"] * c["N"] < 1.5e8:
            return c


# ---- inputs -----------------------------------------------------------------


def _rand(shape, gen, scale=1.0, dtype=torch.bfloat16):
    """Normal values; drawn in slices, so that large weights need no 32-bit copy."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i : i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(scale))
    return out


def _logits(T, E, gen, pad=0.0):
    """A router's logits: some experts are liked more than others; padding rows are all -inf."""
    x = torch.randn(T, E, generator=gen, device="cuda") + 0.7 * torch.randn(1, E, generator=gen, device="cuda")
    x[torch.rand(T, generator=gen, device="cuda") < pad] = -math.inf
    return x


def _order(ids, E):
    """(offsets, rows, slots) of int expert numbers [T, k]; -1 marks an entry without an expert."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    by = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=ids.device), counts[:E].cumsum(0)])
    routed = torch.arange(T * k, device=ids.device) < offsets[E]
    rows = torch.where(routed, by // k, -1)
    slots = torch.empty_like(flat).scatter_(0, by, torch.where(routed, torch.arange(T * k, device=ids.device), -1))
    return offsets.int(), rows.int(), slots.view(T, k).int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T, k = case["op"], case["T"], case["k"]
    s = {"case": case}
    if op == "route":
        x = _logits(T, case["E"], gen, case["pad"])
        s["logits"] = x if case["fp32"] else x.bfloat16()
    elif op in ("up", "down"):
        E, K, N = case["E"], case["K"], case["N"]
        ids = torch.sort(_logits(T, E, gen), dim=1, descending=True, stable=True).indices[:, :k]
        s["offsets"], s["rows"], _ = _order(ids, E)
        counts = s["offsets"][1:] - s["offsets"][:-1]
        # the plain form's plan: each row's expert and its place in that expert's padded block
        s["expert"] = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
        s["place"] = torch.arange(T * k, device="cuda") - s["offsets"].long()[s["expert"]]
        s["most"] = int(counts.max())
        if op == "up":
            s["A"] = _rand((T, K), gen)
            s["W1"], s["W2"] = _rand((E, K, N), gen, K**-0.5), _rand((E, K, N), gen, K**-0.5)
        else:
            s["X"] = _rand((T * k, K), gen, 0.5)
            s["W"] = _rand((E, K, N), gen, K**-0.5)
    else:
        D = case["D"]
        s["R"] = _rand((T, D), gen, 2.0, torch.float32 if case["fp32"] else torch.bfloat16)
        s["Z"] = _rand((T * max(k, 1), D), gen, 0.7)
        s["slots"] = s["weights"] = s["gate"] = None
        if k:
            s["slots"] = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
            s["weights"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), dim=1)
        if case["gate"] != "none":
            s["gate"] = _rand((D,) if case["gate"] == "vector" else (T, D), gen, 0.3)
        s["post"], s["pre"] = (1 + 0.1 * _rand((D,), gen).float()).bfloat16(), (1 + 0.1 * _rand((D,), gen).float()).bfloat16()
        s["scale"] = 0.9375
    return s


# ---- the operators -----------------------------------------------------------


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, : c["k"]], ids[:, : c["k"]]
    chosen = top > -math.inf
    e = torch.exp(top - x.amax(dim=1, keepdim=True))
    e = torch.where(chosen, e, 0.0)
    total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - x.amax(dim=1, keepdim=True)).sum(1, keepdim=True)
    weights = torch.where(chosen, e / total, 0.0)
    ids = torch.where(chosen, ids, -1).int()
    offsets, rows, slots = _order(ids, c["E"])
    return {"ids": ids, "weights": weights, "offsets": offsets, "rows": rows, "slots": slots}


def _plain_products(s, X, weights):
    """X [P, K] times each row's expert's matrix, for each of `weights` [E, K, N], in 32 bits."""
    e, P = s["expert"], X.shape[0]
    if P <= s["case"]["E"]:  # few rows: each takes its own expert's matrix
        return [torch.bmm(X.float().unsqueeze(1), W[e].float()).squeeze(1) for W in weights]
    at = e * s["most"] + s["place"]
    block = torch.zeros(s["case"]["E"] * s["most"], X.shape[1], device=X.device)
    block[at] = X.float()
    block = block.view(s["case"]["E"], s["most"], -1)
    return [torch.bmm(block, W.float()).flatten(0, 1)[at] for W in weights]


def _plain_up(s):
    g, u = _plain_products(s, s["A"][s["rows"].long()], [s["W1"], s["W2"]])
    return (g / (1 + torch.exp(-g)) * u).bfloat16()


def _plain_down(s):
    return _plain_products(s, s["X"], [s["W"]])[0].bfloat16()


def _plain_norm(s):
    z = s["Z"].float()
    if s["slots"] is not None:
        z = (s["weights"].unsqueeze(2) * z[s["slots"].long()]).sum(1)
    z = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        z = s["gate"].float() * z
    r = s["scale"] * s["R"].float() + z
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["pre"].float()
    return {"R": r.to(s["R"].dtype), "H": h.bfloat16()}


def run(state):
    s = state
    op, c = s["case"]["op"], s["case"]
    if not own:
        return {"route": _plain_route, "up": _plain_up, "down": _plain_down, "norm": _plain_norm}[op](s)
    import swiglu_gemm_transformer_gb300 as sg

    if op == "route":
        r = sg.swiglu_moe_route(s["logits"], c["k"], renormalize=c["renorm"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    if op == "up":
        return sg.swiglu_fused_grouped(s["A"], s["W1"], s["W2"], s["offsets"], s["rows"])
    if op == "down":
        return sg.swiglu_linear_grouped(s["X"], s["W"], s["offsets"])
    R, H = sg.swiglu_residual_norm(s["Z"], s["R"], slots=s["slots"], weights=s["weights"], gamma_post=s["post"], gate=s["gate"],
                                   residual_scale=s["scale"], gamma_pre=s["pre"], eps=EPS)
    return {"R": R, "H": H}


def work(case):
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        E, P = case["E"], T * k
        return {"bytes": T * E * (4 if case["fp32"] else 2) + 16 * P + 4 * (E + 1), "flops": 4 * T * E}
    if op == "norm":
        D, P = case["D"], T * max(k, 1)
        gate = {"none": 0, "vector": D, "rows": T * D}[case["gate"]]
        return {"bytes": 2 * P * D + 8 * T * k + 2 * T * D * (4 if case["fp32"] else 2) + 2 * T * D + 2 * gate + 4 * D,
                "flops": 2 * T * k * D + 10 * T * D}
    E, K, N, P = case["E"], case["K"], case["N"], T * k
    # the experts that get rows, as a mean over routers without preference
    used = E * (1 - (1 - k / E) ** T)
    mats = 2 if op == "up" else 1
    return {"bytes": int(2 * mats * used * K * N + 2 * (T if op == "up" else P) * K + 2 * P * N + 4 * (E + 1) + (4 * P if op == "up" else 0)),
            "flops": 2 * mats * P * K * N}


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op, T, k = case["op"], case["T"], case["k"]
    if op == "route":
        x = s["logits"].double()
        there = torch.isfinite(x)
        p = torch.where(there, torch.exp(torch.where(there, x, 0.0)), 0.0)  # logits of a few units: no shift is needed
        # the k largest, ties to the lowest number: rank by how many come before
        w = torch.zeros(T, k, dtype=torch.double, device=x.device)
        left, rank = p.clone(), torch.arange(T, device=x.device)
        for j in range(k):
            e = left.argmax(1)
            w[:, j] = left[rank, e]
            left[rank, e] = 0
        total = w.sum(1, keepdim=True) if case["renorm"] else p.sum(1, keepdim=True)
        return {"ids": None, "weights": torch.where(total > 0, w / total, 0.0), "offsets": None, "rows": None, "slots": None}
    if op in ("up", "down"):
        P, N, off = T * k, case["N"], s["offsets"].tolist()
        out = torch.empty(P, N, dtype=torch.double, device="cuda")
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            if op == "up":
                x = s["A"][s["rows"][a:b].long()].double()
                g = x @ s["W1"][e].double()
                out[a:b] = g * torch.sigmoid(g) * (x @ s["W2"][e].double())
            else:
                out[a:b] = s["X"][a:b].double() @ s["W"][e].double()
        return out
    z = s["Z"].double()
    if s["slots"] is not None:
        z = torch.einsum("tk,tkd->td", s["weights"].double(), z[s["slots"].long()])
    n = z / torch.sqrt(z.square().mean(1, keepdim=True) + EPS) * s["post"].double()
    r = s["scale"] * s["R"].double() + (n if s["gate"] is None else n * s["gate"].double())
    return {"R": r, "H": r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * s["pre"].double()}
