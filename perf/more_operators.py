"""Cases of the sparse SwiGLU layer in 8-bit integers: routing by scores with a
bias and groups, quantisation by rows, and the products in 8-bit integers,
grouped by expert and dense.

For each case ``run`` computes one operator, either in a plain form
(elementary torch operations in 32 bits, the router's choice in 64 because
neighbouring scores may lie closer than 32 bits tell, rounded once at the end)
or through the library's own entry point.  ``exact`` gives the same outputs
from the definitions in 64 bits.

    route   s = sigmoid(l) or softmax(l), c = s + b; the groups with the best
            two (or one) c, the k largest c in them; weights s, their order
    quant   s[r] = max |x[r]| / 127, q = round(127 x / max |x[r]|), returned as s q
    up      Y[p] = SiLU(sa g) * (sa u),  g, u = A[rows[p]] W1[e]^T s1[e], ... W2 ...
    down    Z[p] = sx[p] X[p] W[e]^T sw[e]
    fused, linear   the same for one matrix
"""
import math

import torch

own = False


# ---- cases -----------------------------------------------------------------


def listed():
    return [
        # one token of a serving loop, softmax scores, groups by their best expert: pure latency
        {"name": "route-token", "op": "route", "T": 1, "E": 160, "k": 6, "groups": 8, "kept": 3, "best": 1, "score": "softmax", "bias": False,
         "fp32": False, "renorm": False, "pad": 0.0},
        # a long prompt batch through 256 experts in 8 groups, some rows padding (every logit -inf)
        {"name": "route-prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "groups": 8, "kept": 4, "best": 2, "score": "sigmoid", "bias": True,
         "fp32": True, "renorm": True, "pad": 0.03},
        # the gate/up outputs of a few tokens before the down product
        {"name": "quant-batch", "op": "quant", "R": 61, "K": 1032, "fp32": False},
        # the same of a long prompt, 8 experts a token
        {"name": "quant-prompt", "op": "quant", "R": 65536, "K": 1024, "fp32": False},
        # one token through fine-grained experts: a stream of 8 experts' weights
        {"name": "up-token", "op": "up", "T": 1, "E": 64, "k": 8, "K": 2048, "N": 1024},
        # a long prompt through the same, about 1000 rows an expert
        {"name": "up-prompt", "op": "up", "T": 8192, "E": 64, "k": 8, "K": 2048, "N": 1024},
        # a decode batch of odd size: nearly every expert gets a few rows
        {"name": "down-batch", "op": "down", "T": 61, "E": 64, "k": 8, "K": 1024, "N": 2048},
        {"name": "down-prompt", "op": "down", "T": 8192, "E": 64, "k": 8, "K": 1024, "N": 2048},
        # the 7B projection: one token, and a prompt of odd length
        {"name": "fused-7b-token", "op": "fused", "M": 1, "K": 3584, "N": 18944},
        {"name": "fused-7b-prompt", "op": "fused", "M": 2047, "K": 3584, "N": 18944},
        # the 0.5B down projection for a batch of sequences, and the 72B one for a prompt
        {"name": "linear-0.5b-batch", "op": "linear", "M": 125, "K": 4864, "N": 896},
        {"name": "linear-72b-prompt", "op": "linear", "M": 4095, "K": 29568, "N": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "quant", "up", "down", "fused", "linear"])
    if op == "route":
        per, groups = rng.choice([4, 8, 16, 20, 32]), rng.choice([1, 2, 4, 8])
        kept = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 16384), "E": per * groups, "k": rng.randint(1, min(8, per * kept)), "groups": groups, "kept": kept,
                "best": rng.choice([1, 2]), "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "fp32": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "pad": rng.choice([0.0, 0.1])}
    if op == "quant":
        while True:
            c = {"op": op, "R": _log(rng, 1, 65536), "K": 8 * _log(rng, 16, 2368), "fp32": rng.random() < 0.3}
            if c["R"] * c["K"] < 6.7e7:
                return c
    while True:
        c = {"op": op, "K": 16 * _log(rng, 32, 512), "N": 8 * _log(rng, 64, 2048)}
        if op in ("up", "down"):
            c["T"], c["E"] = _log(rng, 1, 8192), rng.choice([4, 8, 16, 32, 64])
            c["k"] = rng.randint(1, min(8, c["E"]))
            fits = c["E"] * c["K"] * c["N"] < 3e8 and c["T"] * c["k"] * c["K"] * c["N"] < 2e11 and c["T"] * c["k"] * c["N"] < 1.5e8
        else:
            c["M"] = _log(rng, 1, 4096)
            fits = c["M"] * c["K"] * c["N"] < 3e11
        if fits:
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


def _codes(rows, K, gen, scale=1.0):
    """Quantised normal rows: (codes int8 [rows, K], scales [rows]); a few of the columns are larger than the others."""
    q, s = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    loud = 1 + 5 * (torch.rand(K, generator=gen, device="cuda") < 0.01)
    step = max(1, (1 << 26) // K)
    for i in range(0, rows, step):
        x = torch.randn(min(step, rows - i), K, generator=gen, device="cuda").mul_(loud).mul_(scale)
        s[i : i + step] = x.abs().amax(1) / 127
        q[i : i + step] = torch.round(x / s[i : i + step, None]).clamp(-127, 127).to(torch.int8)
    return q, s


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
    op = case["op"]
    s = {"case": case}
    if op == "route":
        x = _logits(case["T"], case["E"], gen, case["pad"])
        s["logits"] = x if case["fp32"] else x.bfloat16()
        s["bias"] = 0.1 * torch.randn(case["E"], generator=gen, device="cuda") if case["bias"] else None
        return s
    if op == "quant":
        s["X"] = _rand((case["R"], case["K"]), gen, 2.0, torch.float32 if case["fp32"] else torch.bfloat16)
        return s
    K, N = case["K"], case["N"]
    if op in ("fused", "linear"):
        s["A"], s["a"] = _codes(case["M"], K, gen)
        s["W"] = [_codes(N, K, gen, K**-0.5) for _ in range(2 if op == "fused" else 1)]
        return s
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.sort(_logits(T, E, gen), dim=1, descending=True, stable=True).indices[:, :k]
    s["offsets"], s["rows"], _ = _order(ids, E)
    counts = s["offsets"][1:] - s["offsets"][:-1]
    # the plain form's plan: each row's expert and its place in that expert's padded block
    s["expert"] = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
    s["place"] = torch.arange(T * k, device="cuda") - s["offsets"].long()[s["expert"]]
    s["most"] = int(counts.max())
    s["A"], s["a"] = _codes(T if op == "up" else T * k, K, gen)
    s["W"] = [(q.view(E, N, K), w.view(E, N)) for q, w in (_codes(E * N, K, gen, K**-0.5) for _ in range(2 if op == "up" else 1))]
    return s


# ---- the operators -----------------------------------------------------------


def _plain_route(s):
    c, x, b = s["case"], s["logits"].double(), s["bias"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    there = x > -math.inf
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - torch.where(there, x, -1e30).amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    score = torch.where(there, score, 0.0)
    worth = torch.where(there, score if b is None else score + b.double(), -math.inf)
    if c["kept"] < G:
        top = torch.sort(worth.view(T, G, E // G), dim=2, descending=True, stable=True).values
        group = top[:, :, 0]
        if c["best"] == 2:
            group = group + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], 0.0)
        best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        worth = torch.where(keep.repeat_interleave(E // G, dim=1), worth, -math.inf)
    top, ids = torch.sort(worth, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    w = torch.where(chosen, score.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    ids = torch.where(chosen, ids, -1).int()
    offsets, rows, slots = _order(ids, E)
    return {"ids": ids, "weights": (2.5 * w).float(), "offsets": offsets, "rows": rows, "slots": slots}


def _plain_quant(s):
    x = s["X"].float()
    most = x.abs().amax(1, keepdim=True)
    q = torch.round(127 * x.double() / most.double())  # half-way values, which 127 x / most often is, need the 64 bits
    scale = most / 127
    return {"values": torch.where(most > 0, q, 0.0).float() * scale, "scale": scale.squeeze(1)}


def _plain_products(s, X):
    """X [P, K] times each row's expert's matrix, for each matrix, in 32 bits, with both scales but the rows'."""
    if "expert" not in s:
        return [X @ q.float().t() * w for q, w in s["W"]]
    e, P, E = s["expert"], X.shape[0], s["case"]["E"]
    if P <= E:  # few rows: each takes its own expert's matrix
        return [torch.bmm(q[e].float(), X.unsqueeze(2)).squeeze(2) * w[e] for q, w in s["W"]]
    at = e * s["most"] + s["place"]
    block = torch.zeros(E * s["most"], X.shape[1], device=X.device)
    block[at] = X
    block = block.view(E, s["most"], -1)
    return [(torch.bmm(block, q.float().transpose(1, 2)) * w.unsqueeze(1)).flatten(0, 1)[at] for q, w in s["W"]]


def _plain_product(s):
    at = s["rows"].long() if s["case"]["op"] == "up" else slice(None)
    a = s["a"][at].unsqueeze(1)
    y = [a * z for z in _plain_products(s, s["A"][at].float())]
    return (y[0] if len(y) == 1 else y[0] / (1 + torch.exp(-y[0])) * y[1]).bfloat16()


def run(state):
    s = state
    op, c = s["case"]["op"], s["case"]
    if not own:
        return {"route": _plain_route, "quant": _plain_quant}.get(op, _plain_product)(s)
    import swiglu_gemm_transformer_gb300 as sg

    if op == "route":
        r = sg.swiglu_moe_route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], kept_groups=c["kept"],
                                       group_best=c["best"], renormalize=c["renorm"], scale=2.5)
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    if op == "quant":
        q, scale = sg.swiglu_quant_int8(s["X"])
        return {"values": q * scale[:, None], "scale": scale}
    (W1, s1), (W2, s2) = s["W"][0], s["W"][-1]
    if op == "up":
        return sg.swiglu_fused_grouped_int8(s["A"], s["a"], W1, s1, W2, s2, s["offsets"], s["rows"])
    if op == "down":
        return sg.swiglu_linear_grouped_int8(s["A"], s["a"], W1, s1, s["offsets"])
    if op == "fused":
        return sg.swiglu_fused_int8(s["A"], s["a"], W1, s1, W2, s2)
    return sg.swiglu_linear_int8(s["A"], s["a"], W1, s1)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, P = case["T"], case["E"], case["T"] * case["k"]
        return {"bytes": T * E * (4 if case["fp32"] else 2) + 4 * E * case["bias"] + 16 * P + 4 * (E + 1), "flops": 8 * T * E}
    if op == "quant":
        R, K = case["R"], case["K"]
        return {"bytes": R * K * ((4 if case["fp32"] else 2) + 4) + 4 * R, "flops": 3 * R * K}  # the values are returned in 32 bits
    K, N = case["K"], case["N"]
    mats = 2 if op in ("up", "fused") else 1
    if op in ("fused", "linear"):
        M = case["M"]
        return {"bytes": K * (M + mats * N) + 4 * (M + mats * N) + 2 * M * N, "flops": 2 * mats * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    P, X = T * k, T if op == "up" else T * k
    # the experts that get rows, as a mean over routers without preference
    used = E * (1 - (1 - k / E) ** T)
    return {"bytes": int(mats * used * N * (K + 4) + X * (K + 4) + 2 * P * N + 4 * (E + 1) + (4 * P if op == "up" else 0)),
            "flops": 2 * mats * P * K * N}


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
        x = s["logits"].double()
        there = torch.isfinite(x)
        x = torch.where(there, x, 0.0)
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.exp(x - torch.logsumexp(torch.where(there, x, -math.inf), 1, keepdim=True))
        p = torch.where(there, p, 0.0)
        c = p + (s["bias"].double() if case["bias"] else 0.0)
        low = torch.full_like(c, -1e9)
        c = torch.where(there, c, low)
        rank = torch.arange(T, device=x.device)
        if case["kept"] < G:
            g = c.view(T, G, E // G)
            first = g.amax(2)
            if case["best"] == 2:
                rest = g.scatter(2, g.argmax(2, keepdim=True), -1e9).amax(2)
                first = first + torch.where(rest > -1e8, rest, 0.0)
            keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
            for _ in range(case["kept"]):
                e = first.argmax(1)
                keep[rank, e] = True
                first[rank, e] = -4e9
            c = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), c, low)
        w = torch.zeros(T, k, dtype=torch.double, device=x.device)
        for j in range(k):
            e = c.argmax(1)
            w[:, j] = torch.where(c[rank, e] > -1e8, p[rank, e], 0.0)
            c[rank, e] = -2e9
        if case["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0.0)
        return {"ids": None, "weights": 2.5 * w, "offsets": None, "rows": None, "slots": None}
    if op == "quant":
        x = s["X"].double()
        top = torch.maximum(x.amax(1), -x.amin(1)).unsqueeze(1)
        y = 127 * x / top
        q = torch.floor(y)  # to the nearest, half-way values to the even one
        q = q + ((y - q > 0.5) | ((y - q == 0.5) & (q % 2 != 0)))
        return {"values": q * top / 127, "scale": top.squeeze(1) / 127}
    M = case["M"] if op in ("fused", "linear") else case["T"] * case["k"]
    if M * case["K"] * case["N"] * len(s["W"]) > 4e12:
        return None  # minutes in 64 bits
    off = s["offsets"].tolist() if "offsets" in s else [0, M]
    out = torch.empty(M, case["N"], dtype=torch.double, device="cuda")
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        at = s["rows"][a:b].long() if op == "up" else slice(a, b)
        x = s["A"][at].double() * s["a"][at].double()[:, None]
        y = [x @ (q if q.dim() == 2 else q[e]).double().t() * (w if w.dim() == 1 else w[e]).double() for q, w in s["W"]]
        out[a:b] = y[0] if len(y) == 1 else y[0] * torch.sigmoid(y[0]) * y[1]
    return out
