"""GPU tests of the router by scores against a plain 64-bit implementation
(written here; no code shared with the library).

Integers are exact.  Weights: an FP32 score is off by 2 units of exp, its
argument's rounding (softmax: |x - m| 2^-24), a sum and a quotient; softmax's
sum has E / 32 + 5 additions; renormalising adds up to 32 scores and one more
quotient, the scale one product: (span + E / 32 + 32) 2^-24 in all, relative.
"""
import math
import zlib

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    import __graft_entry__
    __graft_entry__.build()
    import swiglu_gemm_transformer_gb300 as m
    m.lib()
    return m


def _gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def reference(x, b, k, score, groups, kept, best, renorm, scale):
    """x [T,E], b [E] or None: float64 numpy."""
    T, E = x.shape
    ids, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    first = lambda v: (not math.isnan(v), -v if not math.isnan(v) else 0.0)  # noqa: E731
    with np.errstate(all="ignore"):
        for t in range(T):
            row = x[t]
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-row))
            else:
                there = row[row != -np.inf]
                m = (np.nan if np.isnan(there).any() else there.max()) if there.size else 0.0
                s = np.exp(row - m)
                s = s / s[row != -np.inf].sum()
            c = s if b is None else s + b
            order = row if b is None else c  # the scores' order is the logits'
            ok = (row != -np.inf) & (c != -np.inf)
            value = []
            for g in range(groups):
                mine = [e for e in range(g * E // groups, (g + 1) * E // groups) if ok[e]]
                mine.sort(key=lambda e: (*first(order[e]), e))
                if not mine:
                    value.append(None)
                elif best == 1:
                    value.append(order[mine[0]])
                else:
                    value.append(sum(c[e] for e in mine[:2]))
            left = sorted((g for g in range(groups) if value[g] is not None), key=lambda g: (*first(value[g]), g))[:kept]
            if kept == groups:
                left = range(groups)
            cand = [e for g in left for e in range(g * E // groups, (g + 1) * E // groups) if ok[e]]
            cand.sort(key=lambda e: (*first(order[e]), e))
            cand = cand[:k]
            total = sum(s[e] for e in cand)
            for j, e in enumerate(cand):
                ids[t, j] = e
                w[t, j] = scale * s[e] * (1.0 if not renorm else 0.0 if total == 0 else 1 / total)
    return ids, w


def order_of(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    order = [i for i in np.argsort(np.where(flat < 0, E, flat), kind="stable") if flat[i] >= 0]
    offsets = np.concatenate([[0], np.bincount(flat[flat >= 0], minlength=E).cumsum()])
    rows, slots = np.full(T * k, -1), np.full(T * k, -1)
    rows[: len(order)] = [i // k for i in order]
    slots[order] = np.arange(len(order))
    return offsets, rows, slots.reshape(T, k)


def check(sg, x, k, b=None, *, score="sigmoid", groups=1, kept=None, best=2, renorm=True, scale=2.5, **kw):
    T, E = x.shape
    kept = groups if kept is None else kept
    r = sg.swiglu_moe_route_scored(x.to(DEV), k, score=score, bias=None if b is None else b.to(DEV), groups=groups,
                                   kept_groups=kept, group_best=best, renormalize=renorm, scale=scale, **kw)
    ids, w = reference(x.double().numpy(), None if b is None else b.double().numpy(), k, score, groups, kept, best, renorm, scale)
    np.testing.assert_array_equal(r.ids.cpu().numpy(), ids)
    for got, want in zip((r.offsets, r.rows, r.slots), order_of(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    got = r.weights.double().cpu().numpy()
    nan = np.isnan(w)
    np.testing.assert_array_equal(np.isnan(got), nan)
    there = x[torch.isfinite(x)]
    span = float(there.max() - there.min()) if there.numel() and score == "softmax" else 0.0
    assert (np.abs(got - w)[~nan] <= ((span + E / 32 + 32) * 2.0**-24 * np.abs(w) + 1e-37)[~nan]).all()
    return r


SCORES = pytest.mark.parametrize("score", ["sigmoid", "softmax"])
BIAS = pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])


@SCORES
@BIAS
@pytest.mark.parametrize("shape", [(1, 256, 8, 8, 4, 2), (1, 1, 1, 1, 1, 1), (1, 160, 6, 8, 3, 1), (3, 8, 4, 2, 1, 2), (61, 64, 8, 1, 1, 2),
                                   (128, 72, 5, 8, 2, 2), (300, 256, 8, 8, 4, 2), (257, 96, 32, 32, 16, 2), (40, 1024, 32, 16, 4, 1),
                                   (5, 1024, 9, 32, 3, 2), (500, 20, 3, 4, 4, 2), (33, 512, 8, 1, 1, 1), (1000, 16, 2, 16, 5, 2)],
                         ids=lambda s: "x".join(map(str, s)))
def test_choices(sg, shape, score, bias):
    T, E, k, groups, kept, best = shape
    g = _gen("scored", *shape, score, bias)
    x = torch.randn(T, E, generator=g) * 1.5
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    check(sg, x, k, b, score=score, groups=groups, kept=kept, best=best, renorm=bool(T & 1))
    check(sg, x.to(BF), k, b, score=score, groups=groups, kept=kept, best=best, renorm=bool(E & 4), scale=1.0)


@pytest.mark.parametrize("T", [2, 7, 8, 9, 16, 17, 32, 33, 63, 64, 65, 129, 255, 256])
def test_calls_of_one_launch(sg, T):
    """Blocks of 8 to 32 tokens, full and ragged, some without a token."""
    x = torch.randn(T, 300, generator=_gen("one", T))
    x[T // 2] = -math.inf
    b = torch.randn(300, generator=_gen("oneb")) * 0.1
    check(sg, x, 5, b, groups=4, kept=2)


@SCORES
@pytest.mark.parametrize("best", [1, 2])
def test_ties_go_to_the_lowest(sg, score, best):
    x = torch.randint(-2, 2, (200, 64), generator=_gen("ties", score, best)).float()
    x[0] = 0.5
    check(sg, x, 8, score=score, groups=8, kept=3, best=best)
    check(sg, x, 8, torch.zeros(64), score=score, groups=8, kept=3, best=best)
    check(sg, x, 8, torch.tensor([0.25, -0.5]).repeat(32), score=score, groups=4, kept=2, best=best)


@SCORES
@pytest.mark.parametrize("T,E", [(40, 64), (700, 64), (30, 512)])
def test_choices_closer_than_fp32_tells(sg, score, T, E):
    """Biases that make the scores of a token equal up to FP32's last bits, for every token."""
    g = _gen("close", score, T)
    row = torch.randn(E, generator=g)
    s = torch.sigmoid(row.double()) if score == "sigmoid" else torch.softmax(row.double(), 0)
    b = (1.0 - s).float()  # every c is 1 within 2^-25: FP64 alone orders them
    x = row.repeat(T, 1)
    check(sg, x, 8, b, score=score)
    check(sg, x, 8, b, score=score, groups=8, kept=3, best=2)
    check(sg, x, 8, b, score=score, groups=8, kept=3, best=1)


@SCORES
def test_sums_of_two_scores_closer_than_fp32_tells(sg, score):
    x = torch.randn(300, 32, generator=_gen("sums", score)).to(BF).float()
    x[:, 16:] = x[:, :16].flip(1)  # the groups' two best are alike in pairs: true ties
    x[::3, 3] += 1e-6               # or nearly
    check(sg, x, 4, score=score, groups=8, kept=3, best=2)


@SCORES
@BIAS
@pytest.mark.parametrize("T", [9, 400])
def test_masked(sg, score, bias, T):
    x = torch.randn(T, 48, generator=_gen("mask", score, T))
    b = torch.randn(48, generator=_gen("maskb")) * 0.3 if bias else None
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    x[2, ::2] = -math.inf
    x[3, :12] = -math.inf              # a group without experts
    x[4, 1:12] = x[4, 13:24] = -math.inf  # groups of one
    x[5] = torch.finfo(torch.float32).min
    x[T - 1, 24:] = -math.inf
    for groups, kept, best in ((1, 1, 2), (4, 2, 2), (4, 2, 1), (4, 1, 2)):
        check(sg, x, 6, b, score=score, groups=groups, kept=kept, best=best)


def test_an_expert_switched_off_by_its_bias(sg):
    x = torch.randn(50, 32, generator=_gen("off"))
    for off in (-math.inf, -1e9):
        b = torch.randn(32, generator=_gen("offb")) * 0.1
        b[[0, 5, 6, 7, 31]] = off
        r = check(sg, x, 4, b, groups=8, kept=4)
        assert not (r.ids.cpu()[..., None] == torch.tensor([0, 5, 6, 7, 31])).any()


def test_sigmoids_far_from_zero(sg):
    g = _gen("far")
    x = torch.randn(64, 32, generator=g) * 40
    x[0] = torch.linspace(-120, -89, 32)   # FP32 scores all underflow
    x[1] = torch.linspace(30, 100, 32)     # or are all one
    x[2] = -800.0                          # FP64 ones too: weights of zero
    check(sg, x, 5, groups=4, kept=2)
    check(sg, x, 5, torch.randn(32, generator=g) * 0.01)


@SCORES
def test_nan_and_inf(sg, score):
    x = torch.randn(40, 32, generator=_gen("nan"))
    x[0, 5] = math.nan
    x[1, 7] = math.inf
    x[2, 3], x[2, 30] = math.nan, -math.nan
    r = check(sg, x, 4, score=score, groups=4, kept=2, best=1)
    assert int(r.ids[0, 0]) == 5 and torch.isnan(r.weights[0, 0])
    assert not torch.isnan(r.weights[3:]).any()


def test_no_tokens(sg):
    r = sg.swiglu_moe_route_scored(torch.empty(0, 8, device=DEV), 2, offsets=torch.full((9,), 7, dtype=torch.int32, device=DEV))
    assert r.offsets.tolist() == [0] * 9 and r.rows.numel() == 0


def test_scores_without_groups_choose_as_the_logits_do(sg):
    x = torch.randn(700, 64, generator=_gen("same")).to(DEV)
    a = sg.swiglu_moe_route(x, 8, renormalize=True)
    b = sg.swiglu_moe_route_scored(x, 8, score="softmax", renormalize=True)
    for i in (0, 2, 3, 4):
        assert torch.equal(a[i], b[i])
    torch.testing.assert_close(a.weights, b.weights, rtol=2e-6, atol=0)


@pytest.mark.parametrize("T", [5, 700])
def test_captured_and_replayed_on_new_logits(sg, T):
    x = torch.zeros(T, 64, device=DEV)
    b = torch.randn(64, generator=_gen("graphb")) * 0.1
    bd = b.to(DEV)
    call = lambda: sg.swiglu_moe_route_scored(x, 4, bias=bd, groups=8, kept_groups=3)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(3):
        new = torch.randn(T, 64, generator=_gen("graph", i))
        x.copy_(new)
        graph.replay()
        ids, _ = reference(new.double().numpy(), b.double().numpy(), 4, "sigmoid", 8, 3, 2, True, 1.0)
        np.testing.assert_array_equal(out.ids.cpu().numpy(), ids)
        for got, want in zip(out[2:], order_of(ids, 64)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_binding_refusals(sg):
    x = torch.zeros(4, 48, device=DEV)
    for kw, err in ((dict(score="tanh"), ValueError), (dict(groups=3), ValueError), (dict(groups=32), ValueError),
                    (dict(groups=4, kept_groups=5), ValueError), (dict(groups=4, kept_groups=0), ValueError),
                    (dict(group_best=3), ValueError), (dict(bias=torch.zeros(47, device=DEV)), ValueError),
                    (dict(bias=torch.zeros(48, dtype=BF, device=DEV)), TypeError), (dict(bias=torch.zeros(48)), ValueError),
                    (dict(groups=16, kept_groups=1, k=4), ValueError), (dict(scale=math.inf), sg.SwigluError)):
        with pytest.raises(err):
            sg.swiglu_moe_route_scored(x, **{"k": 2, **kw})
    with pytest.raises(ValueError):
        sg.swiglu_moe_route_scored(x, 0)
    with pytest.raises(ValueError):
        sg.swiglu_moe_route_scored(x.t(), 2)


@SCORES
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("pin", [math.inf, math.nan], ids=["inf", "nan"])
@pytest.mark.parametrize("T,E", [(40, 32), (300, 64), (20, 512)])
def test_a_pinned_expert_keeps_its_group_where_other_groups_are_close(sg, score, best, pin, T, E):
    """Experts of a bias of +inf, one to three of them, beside groups whose values FP64 alone tells apart."""
    row = torch.randn(E, generator=_gen("pinned", E))
    s = torch.sigmoid(row.double()) if score == "sigmoid" else torch.softmax(row.double(), 0)
    x = row.repeat(T, 1)
    x[1::4] = torch.randn(len(x[1::4]), E, generator=_gen("pinned rows", E))
    size = E // 8
    for pinned in ((5 * size + 1,), (5 * size, 5 * size + 1), (2 * size, 5 * size + 2, 7 * size + 1)):
        b = (1.0 - s).float()
        b[list(pinned)] = pin
        r = check(sg, x, 4, b, score=score, groups=8, kept=3, best=best)
        assert (r.ids.cpu()[:, : len(pinned)] == torch.tensor(pinned)).all()


@pytest.mark.parametrize("bias", [math.inf, math.nan], ids=["inf", "nan"])
def test_more_pinned_experts_than_choices(sg, bias):
    """Equal infinities are ties: the lowest experts."""
    x = torch.randn(70, 64, generator=_gen("many pinned"))
    b = torch.randn(64, generator=_gen("many pinned b")) * 0.1
    b[3::5] = bias
    for groups, kept, best in ((1, 1, 2), (8, 3, 1), (8, 3, 2)):
        check(sg, x, 6, b, groups=groups, kept=kept, best=best)
    check(sg, x, 6, torch.full((64,), bias), groups=8, kept=3)


@SCORES
@pytest.mark.parametrize("shape", [(300, 1024, 8, 8, 4, 2), (257, 1022, 6, 2, 1, 1), (600, 513, 3, 1, 1, 2), (700, 70, 5, 2, 2, 2),
                                   (5000, 33, 4, 1, 1, 1)], ids=lambda s: "x".join(map(str, s)))
def test_two_launches_of_many_or_odd_experts(sg, shape, score):
    """Blocks of fewer warps, and counts that are no whole pieces of four experts."""
    T, E, k, groups, kept, best = shape
    g = _gen("two launches", *shape, score)
    x = torch.randn(T, E, generator=g) * 1.5
    x[T // 3] = -math.inf
    check(sg, x, k, torch.randn(E, generator=g) * 0.1, score=score, groups=groups, kept=kept, best=best)
