"""GPU tests of the sparse MLP block's operators against plain 64-bit
implementations (written here; no code shared with the library).

Tolerances, derived from the arithmetic:
  * grouped products: the kernel adds K products in FP32, so a sum is off by at
    most K 2^-23 S, S = sum |a| |w| (2^-23 a term covers truncating adders);
    the result is rounded once to BF16 (at most 2^-9 relative; 2^-8 is allowed,
    a result next to a binade's end included).  For SiLU(g) u that error of g
    and u enters with |d SiLU| <= 1.1 and the fast exp and divide with 2^-19.
  * routing weights: expf is within 2 units, its argument within |x - m| 2^-24,
    the sum of E terms within (E / 32 + 5) 2^-24, the divide and the scale
    within 2^-23: together (|x - m| + E / 32 + 16) 2^-24, relative.  Integers
    are exact.
  * norms: each output is a sum of terms with a few roundings and a root mean
    square whose sum of squares has at most 48 roundings in a row: 128 2^-24 of
    the sum of the terms' magnitudes, plus the rounding to BF16 where it is
    BF16.
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


def _status(sg):
    rc, detail = sg.swiglu_device_status()
    assert rc == sg.OK, f"device status {sg.status_string(rc)} detail {detail}"


def _gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


# ---- routing ------------------------------------------------------------------


def route_ref(x, k, renorm, scale):
    """Plain routing in 64 bits; x [T,E] float64 numpy."""
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    span = np.zeros((T, k))
    for t in range(T):
        row = x[t]
        key = np.where(np.isnan(row), np.inf, row)
        nan_first = np.where(np.isnan(row), 0, 1)
        order = sorted(range(E), key=lambda e: (nan_first[e], -key[e], e))
        order = [e for e in order if row[e] != -np.inf][:k]
        if not order:
            continue
        with np.errstate(invalid="ignore"):
            m = row[order[0]]
            p = np.exp(row - m)
            total = p[order].sum() if renorm else p.sum()
            for j, e in enumerate(order):
                ids[t, j], w[t, j], span[t, j] = e, scale * p[e] / total, m - row[e]
    flat = ids.reshape(-1)
    order = [i for i in np.argsort(np.where(flat < 0, E, flat), kind="stable") if flat[i] >= 0]
    offsets = np.zeros(E + 1, np.int64)
    for e in flat[flat >= 0]:
        offsets[e + 1] += 1
    offsets = offsets.cumsum()
    rows = np.full(T * k, -1, np.int64)
    slots = np.full(T * k, -1, np.int64)
    for pos, i in enumerate(order):
        rows[pos], slots[i] = i // k, pos
    return ids, w, offsets, rows, slots.reshape(T, k), span


def check_route(sg, logits, k, renorm=False, scale=1.0, **kw):
    T, E = logits.shape
    r = sg.swiglu_moe_route(logits.to(DEV), k, renormalize=renorm, scale=scale, **kw)
    _status(sg)
    ids, w, offsets, rows, slots, span = route_ref(logits.double().numpy(), k, renorm, scale)
    for got, want, name in ((r.ids, ids, "ids"), (r.offsets, offsets, "offsets"), (r.rows, rows, "rows"),
                            (r.slots, slots, "slots")):
        assert got.dtype == torch.int32
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
    got = r.weights.cpu().double().numpy()
    nan = np.isnan(w)
    np.testing.assert_array_equal(np.isnan(got), nan)
    span = np.where(np.isfinite(span), span, 0)
    tol = (span.max(initial=0.0) + E / 32 + 16) * 2.0**-24 * np.abs(w) + 1e-37
    assert (np.abs(got - w)[~nan] <= tol[~nan]).all()
    return r


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("shape", [(1, 64, 8), (1, 1, 1), (3, 4, 4), (16, 8, 2), (17, 33, 3), (127, 60, 6), (128, 64, 8),
                                   (129, 64, 8), (1000, 128, 4), (300, 256, 8), (257, 500, 7), (130, 1024, 32),
                                   (77, 1024, 32), (2049, 16, 1), (33, 64, 8), (256, 64, 8), (257, 8, 8), (4865, 32, 2),
                                   (9729, 12, 3), (40, 600, 9)], ids=lambda s: "x".join(map(str, s)))
def test_route(sg, shape, fp32):
    T, E, k = shape
    x = torch.randn(T, E, generator=_gen("route", *shape)) * 2
    x = x if fp32 else x.to(BF)
    check_route(sg, x, k, renorm=bool(T & 1), scale=1.0 if T & 2 else 2.5)


@pytest.mark.parametrize("T", [5, 200])
def test_route_ties_go_to_the_lowest_expert(sg, T):
    x = torch.randint(-2, 3, (T, 96), generator=_gen("ties", T)).float()
    x[0] = 1.0
    x[1] = 0.0
    check_route(sg, x, 8, renorm=True)


@pytest.mark.parametrize("T", [9, 400, 5000])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masked(sg, T, renorm):
    x = torch.randn(T, 40, generator=_gen("mask", T))
    x[0] = -math.inf                 # nothing left
    x[1, 1:] = -math.inf             # one expert left
    x[2, ::2] = -math.inf
    x[3] = torch.finfo(torch.float32).min   # the lowest finite value is a logit like any other
    x[4, :35] = -math.inf            # five left, six wanted
    x[5, :] = -1e30
    x[T - 1] = -math.inf
    r = check_route(sg, x, 6, renorm=renorm)
    assert (r.ids[0] == -1).all() and (r.slots[0] == -1).all() and (r.weights[0] == 0).all()


def test_route_every_token_masked(sg):
    for T in (4, 300):
        r = check_route(sg, torch.full((T, 16), -math.inf), 4)
        assert int(r.offsets[-1]) == 0 and (r.rows == -1).all()


@pytest.mark.parametrize("T", [8, 300])
def test_route_nan_and_inf_stay_visible(sg, T):
    x = torch.randn(T, 64, generator=_gen("nan", T))
    x[0, 5] = math.nan
    x[1, 7] = math.inf
    x[2, 3], x[2, 60] = -math.nan, math.nan
    x[3, 9], x[3, 2] = math.inf, -math.inf
    r = check_route(sg, x, 4)
    assert torch.isnan(r.weights[0]).all() and int(r.ids[0, 0]) == 5


def test_route_signed_zeros(sg):
    # -0 ranks as +0 does: the lower expert wins
    x = torch.tensor([[-0.0, 0.0, -1.0], [0.0, -0.0, -1.0]])
    r = sg.swiglu_moe_route(x.to(DEV), 2)
    assert r.ids.tolist() == [[0, 1], [0, 1]]


def test_route_empty(sg):
    r = sg.swiglu_moe_route(torch.empty(0, 8, dtype=BF, device=DEV), 2,
                            offsets=torch.full((9,), 7, dtype=torch.int32, device=DEV))
    assert r.offsets.tolist() == [0] * 9 and r.rows.numel() == 0


def test_route_runs_again_into_the_same_buffers_and_on_another_stream(sg):
    s = torch.cuda.Stream()
    out = None
    ws = torch.empty(sg.lib().swiglu_moe_route_workspace_size(700, 64, 8), dtype=torch.uint8, device=DEV)
    for i in range(3):
        x = torch.randn(700, 64, generator=_gen("again", i))
        xd = x.to(DEV)
        s.wait_stream(torch.cuda.current_stream())
        out = sg.swiglu_moe_route(xd, 8, stream=s, workspace=ws, **(out._asdict() if out else {}))
        s.synchronize()
        ids, _, offsets, rows, slots, _ = route_ref(x.double().numpy(), 8, False, 1.0)
        assert (out.ids.cpu().numpy() == ids).all() and (out.rows.cpu().numpy() == rows).all()
        assert (out.offsets.cpu().numpy() == offsets).all() and (out.slots.cpu().numpy() == slots).all()


@pytest.mark.parametrize("stream", [lambda s: s, lambda s: s.cuda_stream], ids=["object", "handle"])
def test_outputs_and_workspaces_belong_to_the_stream_of_the_call(sg, stream):
    """Memory that the current stream has queued work for is not handed to a call
    on another stream, nor the call's workspace to the current stream."""
    T, E, k, N, K = 4096, 64, 8, 256, 128
    s = torch.cuda.Stream()
    gen = _gen("pools")
    lg = torch.randn(T, E, generator=gen).to(DEV)
    A, R = (torch.randn(T, K, generator=gen).to(DEV, BF) for _ in range(2))
    W1, W2 = (torch.randn(E, K, N, generator=gen).div(11).to(DEV, BF) for _ in range(2))
    W3 = torch.randn(E, N, K, generator=gen).div(16).to(DEV, BF)

    def step(**kw):
        r = sg.swiglu_moe_route(lg, k, renormalize=True, **kw)
        y = sg.swiglu_fused_grouped(A, W1, W2, r.offsets, r.rows, **kw)
        z = sg.swiglu_linear_grouped(y, W3, r.offsets, **kw)
        return [*r, y, z, *sg.swiglu_residual_norm(z, R, slots=r.slots, weights=r.weights, **kw)]

    want = [t.cpu() for t in step()]
    sizes = [t.numel() * t.element_size() for t in want] + [sg.lib().swiglu_moe_route_workspace_size(T, E, k)]
    torch.cuda.synchronize()
    # the current stream still has to write to blocks that it has given back
    torch.cuda._sleep(100_000_000)
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x7F)
    got = step(stream=stream(s))
    # the side stream still works with the workspace when the current one asks for memory
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    late = step(stream=stream(s))
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x7F)
    torch.cuda.synchronize()
    _status(sg)
    for w, a, b in zip(want, got, late):
        assert torch.equal(w, a.cpu()) and torch.equal(w, b.cpu())


# ---- grouped products -----------------------------------------------------------


def grouped_ref(A, Ws, offsets, rows):
    """(value, allowed error) per element in 64 bits; NaN where no expert owns the place."""
    P = len(rows) if rows is not None else A.shape[0]
    N, K = Ws[0].shape[2], A.shape[1]
    Ad = A.double()
    ref = torch.full((P, N), math.nan, dtype=torch.double)
    tol = torch.zeros(P, N, dtype=torch.double)
    acc = K * 2.0**-23
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a >= b:
            continue
        if rows is None:
            x = Ad[a:b]
        else:
            r = torch.tensor(rows[a:b])
            ok = (r >= 0) & (r < A.shape[0])
            x = torch.where(ok[:, None], Ad[r.clamp(0, A.shape[0] - 1)], 0.0)
        g = x @ Ws[0][e].double()
        dg = acc * (x.abs() @ Ws[0][e].double().abs())
        if len(Ws) == 1:
            ref[a:b], tol[a:b] = g, dg
        else:
            u = x @ Ws[1][e].double()
            du = acc * (x.abs() @ Ws[1][e].double().abs())
            s = g * torch.sigmoid(g)
            ref[a:b] = s * u
            tol[a:b] = 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0**-19 * (s * u).abs()
    return ref, tol + 2.0**-8 * ref.abs() + 1e-38


SENTINEL = -77.0


def check_grouped(sg, fused, sizes, N, K, T=None, first=0, spare=0, seed=0, edit=None):
    """sizes: rows of each expert; T: rows of A that `rows` draws from (None: no rows)."""
    E = len(sizes)
    gen = _gen("grouped", fused, tuple(sizes), N, K, seed)
    offsets = [first]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    P = offsets[-1] + spare
    A = torch.randn(P if T is None else T, K, generator=gen).to(BF)
    Ws = [(torch.randn(E, K, N, generator=gen) / math.sqrt(max(K, 1))).to(BF) for _ in range(2 if fused else 1)]
    rows = None if T is None else torch.randint(0, T, (P,), generator=gen).tolist()
    if edit:
        edit(A, Ws, rows)
    Y = torch.full((P, N), SENTINEL, dtype=BF, device=DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    rd = None if rows is None else torch.tensor(rows, dtype=torch.int32, device=DEV)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    fn(A.to(DEV), *[W.to(DEV) for W in Ws], off, rd, Y)
    _status(sg)
    ref, tol = grouped_ref(A, Ws, offsets, rows)
    got = Y.double().cpu()
    assert (got[:first] == SENTINEL).all() and (got[offsets[-1]:] == SENTINEL).all()
    body = slice(first, offsets[-1])
    err = (got - ref).abs()[body]
    assert not torch.isnan(got[body]).any()
    bad = err > tol[body]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}, worst {(err / tol[body]).max()}"
    return got


FORMS = pytest.mark.parametrize("fused", [True, False], ids=["fused", "linear"])


@FORMS
@pytest.mark.parametrize("gather", [True, False], ids=["rows", "dense"])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [0, 0, 1, 0], [31, 32, 33], [64, 65, 1, 0, 63], [255, 256, 257, 0, 2],
                                   [700, 0, 0, 1, 513], [127, 128, 129, 97]], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("NK", [(8, 8), (72, 136), (264, 200), (512, 64)], ids=lambda s: "x".join(map(str, s)))
def test_grouped(sg, fused, gather, sizes, NK):
    check_grouped(sg, fused, sizes, *NK, T=53 if gather else None)


@FORMS
def test_grouped_one_row(sg, fused):
    check_grouped(sg, fused, [0, 0, 0, 1], 1024, 2048, T=1)


@FORMS
@pytest.mark.parametrize("E", [1, 2, 31, 32, 33, 64, 257, 1024])
def test_grouped_expert_counts(sg, fused, E):
    g = _gen("experts", E)
    sizes = torch.randint(0, 4, (E,), generator=g).tolist()
    sizes[-1] = 1
    check_grouped(sg, fused, sizes, 40, 24, T=17)


@FORMS
def test_grouped_more_units_than_pairs(sg, fused):
    check_grouped(sg, fused, [300, 17, 0, 520, 64, 1, 129, 33], 2568, 136, T=200)


@FORMS
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_leaves_other_places_alone(sg, fused, gather):
    check_grouped(sg, fused, [3, 0, 40], 136, 72, T=9 if gather else None, first=5, spare=11)


@FORMS
def test_grouped_long_k_wraps_the_ring(sg, fused):
    check_grouped(sg, fused, [2, 0, 33], 64, 4872, T=20)
    check_grouped(sg, fused, [300, 260], 64, 4872, T=20)


@FORMS
@pytest.mark.parametrize("gather", [True, False], ids=["rows", "dense"])
@pytest.mark.parametrize("sizes", [[1, 0], [0, 2, 0, 1], [5, 33, 0, 70], [128, 1], [300], [17, 0, 0, 0, 0, 0, 0, 0, 0, 1]],
                         ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("NK", [(8, 1024), (72, 1032), (264, 1096), (520, 2056), (2600, 1120)], ids=lambda s: "x".join(map(str, s)))
def test_grouped_few_units_share_k(sg, fused, gather, sizes, NK):
    """So few tiles that several pairs share each one's K."""
    check_grouped(sg, fused, sizes, *NK, T=29 if gather else None)


@FORMS
@pytest.mark.parametrize("gather", [True, False], ids=["rows", "dense"])
@pytest.mark.parametrize("E,rows_each,N,K", [(1024, 2, 1024, 24), (16, 1300, 8192, 40)], ids=["short", "long"])
def test_grouped_ring_of_units_wraps(sg, fused, gather, E, rows_each, N, K):
    """More than 64 units a pair (107, and 75 to 82), so that each half of the ring
    of units is filled again, in tiles of up to 128 rows and of up to 256."""
    gen = _gen("ringwrap", fused, gather, E)
    N = N if fused else 2 * N
    sizes = [int(v) for v in torch.randint(rows_each // 2, rows_each * 3 // 2 + 1, (E,), generator=gen)]
    offsets = [0]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    P, T = offsets[-1], 400 if gather else offsets[-1]
    A = torch.randn(T, K, generator=gen).to(BF)
    Ws = [(torch.randn(E, K, N, generator=gen) / math.sqrt(K)).to(BF) for _ in range(2 if fused else 1)]
    rows = torch.randint(0, T, (P,), generator=gen) if gather else None
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    rd = None if rows is None else rows.int().to(DEV)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    Y = fn(A.to(DEV), *[W.to(DEV) for W in Ws], off, rd, torch.full((P, N), math.nan, dtype=BF, device=DEV))
    _status(sg)
    assert not torch.isnan(Y).any()
    got = Y.cpu()
    for e in range(0, E, max(1, E // 100)):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        pick = torch.arange(a, b)[torch.randperm(b - a, generator=gen)[:24]]
        x = A[pick if rows is None else rows[pick]]
        ref, tol = grouped_ref(x, [W[e:e + 1] for W in Ws], [0, len(pick)], None)
        assert ((got[pick].double() - ref).abs() <= tol).all(), e


def test_grouped_many_long_units_within_a_short_limit(sg):
    """The finder of the units waits for 32 of them at a time: about 2.7 ms here,
    where one takes 0.08 ms, so a limit of 1.5 ms (a wait may take 1 ms or more) is
    kept by every wait of its own and must not end this one."""
    P, K, N = 85000, 16384, 4096        # 333 row tiles x 16 column tiles: 70 units a pair
    gen = torch.Generator(device="cuda").manual_seed(8)
    X = torch.empty(P, K, dtype=BF, device=DEV)
    for a in range(0, P, 5000):
        X[a:a + 5000] = torch.randn(5000, K, generator=gen, device=DEV)
    W = (torch.randn(1, K, N, generator=gen, device=DEV) / 128).to(BF)
    off = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    _status(sg)
    sg.swiglu_set_wait_timeout_ns(1_500_000)
    try:
        Z = sg.swiglu_linear_grouped(X, W, off)
    finally:
        sg.swiglu_set_wait_timeout_ns(2_000_000_000)
    _status(sg)
    for a, b in ((0, 3), (42000, 42002), (P - 3, P)):
        ref, tol = grouped_ref(X[a:b].cpu(), [W.cpu()], [0, b - a], None)
        assert ((Z[a:b].double().cpu() - ref).abs() <= tol).all(), (a, b)


@FORMS
def test_grouped_next_expert_and_other_rows_never_leak(sg, fused):
    """NaN in an expert without rows, and in rows of A that no place names, stay out
    (a ragged K step must not reach into the next expert's matrix)."""
    def edit(A, Ws, rows):
        for W in Ws:
            W[1] = math.nan
        A[7] = math.nan
        for i, r in enumerate(rows):
            if r == 7:
                rows[i] = 6
    check_grouped(sg, fused, [30, 0, 50], 136, 72, T=20, edit=edit)


@FORMS
def test_grouped_nan_row_stays_in_its_row(sg, fused):
    A = torch.randn(40, 64, generator=_gen("nanrow")).to(BF)
    A[11] = math.nan
    Ws = [torch.randn(2, 64, 72, generator=_gen("nanw", i)).to(BF) for i in range(2 if fused else 1)]
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    Y = fn(A.to(DEV), *[W.to(DEV) for W in Ws], off)
    _status(sg)
    bad = torch.isnan(Y).all(1).cpu()
    assert bad[11] and int(bad.sum()) == 1 and int(torch.isnan(Y).any(1).sum()) == 1


@FORMS
def test_grouped_row_numbers_outside_a_give_zeros(sg, fused):
    def edit(A, Ws, rows):
        rows[0], rows[3], rows[35], rows[69] = -1, 20, 1 << 30, -(1 << 31)
    got = check_grouped(sg, fused, [30, 40], 136, 72, T=20, edit=edit)
    assert (got[[0, 3, 35, 69]] == 0).all()


@FORMS
@pytest.mark.parametrize("offsets", [[0, 30, 10, 50], [-5, 10, 20, 90], [40, 30, 20, 10], [60, 60, 60, 60]])
def test_grouped_malformed_offsets_stay_in_bounds(sg, fused, offsets):
    """Offsets are clamped to [0, P] and made monotone."""
    P, K, N = 50, 72, 136
    A = torch.randn(P, K, generator=_gen("mal")).to(BF)
    Ws = [(torch.randn(3, K, N, generator=_gen("malw", i)) / 8).to(BF) for i in range(2 if fused else 1)]
    clean, top = [], 0
    for v in offsets:
        top = max(top, min(max(v, 0), P))
        clean.append(top)
    buf = torch.full((P + 64, N), SENTINEL, dtype=BF, device=DEV)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    fn(A.to(DEV), *[W.to(DEV) for W in Ws], torch.tensor(offsets, dtype=torch.int32, device=DEV), None, buf[:P])
    _status(sg)
    ref, tol = grouped_ref(A, Ws, clean, None)
    got = buf.double().cpu()
    own = slice(clean[0], clean[-1])
    assert ((got[:P][own] - ref[own]).abs() <= tol[own]).all()
    assert (got[:clean[0]] == SENTINEL).all() and (got[clean[-1]:] == SENTINEL).all()


@FORMS
def test_grouped_zero_k_and_no_rows(sg, fused):
    W = torch.empty(2, 0, 16, dtype=BF, device=DEV)
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    Y = fn(torch.empty(5, 0, dtype=BF, device=DEV), *[W] * (2 if fused else 1), off)
    assert (Y == 0).all()
    W = torch.ones(2, 16, 16, dtype=BF, device=DEV)
    Y = fn(torch.empty(0, 16, dtype=BF, device=DEV), *[W] * (2 if fused else 1), torch.zeros_like(off))
    assert Y.shape == (0, 16)


@FORMS
def test_grouped_repeats_bit_for_bit_on_another_stream(sg, fused):
    gen = _gen("stream", fused)
    A = torch.randn(200, 264, generator=gen).to(BF).to(DEV)
    Ws = [(torch.randn(8, 264, 392, generator=gen) / 16).to(BF).to(DEV) for _ in range(2 if fused else 1)]
    r = sg.swiglu_moe_route(torch.randn(200, 8, generator=gen).to(DEV), 3)
    fn = sg.swiglu_fused_grouped if fused else sg.swiglu_linear_grouped
    first = fn(A, *Ws, r.offsets, r.rows)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = [fn(A, *Ws, r.offsets, r.rows, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(first, y) for y in again)


# ---- norms with gate and residual ------------------------------------------------


def norm_ref(Z, R, slots, weights, post, gpost, gate, scale, gpre, eps):
    """(R', H, error allowed of R' and H before their rounding) in 64 bits."""
    z = Z.double()
    mag = z.abs()
    T, D = R.shape
    if slots is not None:
        ok = (slots >= 0) & (slots < Z.shape[0])
        at = slots.clamp(0, max(Z.shape[0] - 1, 0)).long()
        w = torch.where(ok, weights.double(), 0.0)
        zz = torch.where(ok[..., None], z[at], 0.0) if Z.shape[0] else torch.zeros(*slots.shape, D, dtype=torch.double)
        z = (w[..., None] * zz).sum(1)
        mag = (w[..., None] * zz).abs().sum(1)

    def inv(v):
        d = v.square().mean(1, keepdim=True) + eps
        return torch.where(d == 0, 0.0, 1 / torch.sqrt(d))
    f = torch.ones(1, D, dtype=torch.double)
    # the norm's sum of squares takes over z's own error: relative to the rms of the magnitudes
    if post:
        i = inv(z)
        rel = (mag.square().mean(1, keepdim=True).sqrt() * i).clamp(min=1.0)
        f = f * i
        mag = mag + z.abs() * rel
    if gpost is not None:
        f = f * gpost.double()
    if gate is not None:
        f = f * gate.double()
    r = scale * R.double() + z * f
    dr = 128 * 2.0**-24 * ((scale * R.double()).abs() + mag * f.abs())
    i = inv(r)
    g = 1.0 if gpre is None else gpre.double()
    h = r * i * g
    dh = (dr + 128 * 2.0**-24 * r.abs() + r.abs() * i * dr.square().mean(1, keepdim=True).sqrt()) * i * abs(g)
    return r, h, dr, dh


def check_norm(sg, T, D, k=0, r32=False, post=True, gammas=True, gate=None, scale=0.75, eps=1e-6, edit=None, inplace=False):
    gen = _gen("norm", T, D, k, r32)
    P = T * k if k else T
    Z = torch.randn(P, D, generator=gen).to(BF)
    R = torch.randn(T, D, generator=gen) * 2
    R = R if r32 else R.to(BF)
    slots = weights = None
    if k:
        slots = torch.randperm(P, generator=gen).int().view(T, k)
        weights = torch.rand(T, k, generator=gen)
    gp = (1 + 0.2 * torch.randn(D, generator=gen)).to(BF) if gammas and post else None
    gq = (1 + 0.2 * torch.randn(D, generator=gen)).to(BF) if gammas else None
    g = gd = None
    if gate == "vector":
        g = torch.randn(D, generator=gen).to(BF)
        gd = g.to(DEV)
    elif gate == "rows":
        g = torch.randn(T, D, generator=gen).to(BF)
        gd = g.to(DEV)
    elif gate == "strided":
        g = torch.randn(T, 2 * D + 8, generator=gen).to(BF)
        gd = g.to(DEV)[:, 8:D + 8]
        g = g[:, 8:D + 8]
    elif gate == "expanded":
        g = torch.randn(1, D, generator=gen).to(BF).expand(T, D)
        gd = g[:1].to(DEV).expand(T, D)
    if edit:
        edit(Z, R, slots, weights)

    def dev(t):
        return t.to(DEV) if t is not None else None
    Rd = R.to(DEV)
    Ro, H = sg.swiglu_residual_norm(dev(Z), Rd, slots=dev(slots), weights=dev(weights), post_norm=post,
                                    gamma_post=dev(gp), gate=gd, residual_scale=scale, gamma_pre=dev(gq), eps=eps,
                                    Rout=Rd if inplace else None)
    _status(sg)
    r, h, dr, dh = norm_ref(Z, R, slots, weights, post, gp, g, scale, gq, eps)
    assert Ro.dtype == R.dtype and H.dtype == BF
    er = (Ro.double().cpu() - r).abs()
    eh = (H.double().cpu() - h).abs()
    assert (er <= dr + (0 if r32 else 2.0**-8) * r.abs() + 1e-38).all(), (er / (dr + 1e-38)).max()
    assert (eh <= dh + 2.0**-8 * h.abs() + 1e-38).all(), (eh / (dh + 2.0**-8 * h.abs() + 1e-38)).max()
    return Ro, H


@pytest.mark.parametrize("r32", [False, True], ids=["r16", "r32"])
@pytest.mark.parametrize("D", [8, 256, 264, 896, 1024, 2048, 2056, 3584, 4096, 4104, 8192, 8200, 16384, 32768])
def test_norm_widths(sg, D, r32):
    check_norm(sg, 5, D, r32=r32, gate="vector")
    check_norm(sg, 3, D, k=2, r32=r32)


@pytest.mark.parametrize("T", [1, 2, 33, 1000])
@pytest.mark.parametrize("k", [0, 1, 3, 8, 17])
def test_norm_rows_and_joins(sg, T, k):
    check_norm(sg, T, 512, k=k, r32=bool(k & 1), gate="rows")


# more rows than the direct kernel takes: the ring in shared memory
@pytest.mark.parametrize("r32", [False, True], ids=["r16", "r32"])
@pytest.mark.parametrize("D,k", [(8, 0), (256, 1), (512, 0), (520, 3), (1024, 8), (2048, 8), (2056, 2), (4096, 0), (8192, 2),
                                 (8200, 0), (16384, 0), (264, 30), (264, 33)])
def test_norm_many_rows(sg, D, k, r32):
    def edit(Z, R, slots, weights):
        if slots is not None:
            slots[5] = -1
            slots[7, 0] = Z.shape[0] + 3
    check_norm(sg, 701, D, k=k, r32=r32, gate="rows" if D % 16 == 0 else "vector", edit=edit)


def test_norm_weights_of_every_choice_reach_their_row(sg):
    """The shortest rows and the most choices of the ring form: a row's copies take
    the least time that they can, and 30 lanes write a weight each.  Only one
    choice of a row counts, a different one from row to row, and it is exact."""
    T, D, k = 60000, 8, 30
    gen = torch.Generator(device="cuda").manual_seed(9)
    Z = torch.randn(T, D, generator=gen, device=DEV).to(BF)
    at = torch.randint(0, k, (T, 1), generator=gen, device=DEV)
    slots = torch.randint(0, T, (T, k), generator=gen, device=DEV).int()
    weights = torch.zeros(T, k, device=DEV).scatter_(1, at, 1.0 + at.float())
    R = torch.zeros(T, D, device=DEV)
    want = Z[slots.gather(1, at).long().squeeze(1)].float() * (1.0 + at.float())
    for _ in range(20):
        Ro, _ = sg.swiglu_residual_norm(Z, R, slots=slots, weights=weights, post_norm=False)
        assert torch.equal(Ro, want)
    _status(sg)


@pytest.mark.parametrize("gate", [None, "vector", "rows", "strided", "expanded"])
@pytest.mark.parametrize("post", [True, False])
def test_norm_many_rows_forms(sg, gate, post):
    check_norm(sg, 1300, 904, k=2, gate=gate, post=post, gammas=False)
    check_norm(sg, 1300, 904, gate=gate, post=post, r32=True, inplace=True)


@pytest.mark.parametrize("gate", [None, "vector", "rows", "strided", "expanded"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gammas", [True, False])
def test_norm_forms(sg, gate, post, gammas):
    check_norm(sg, 7, 904, k=2, gate=gate, post=post, gammas=gammas)
    check_norm(sg, 7, 904, gate=gate, post=post, gammas=gammas, r32=True)


def test_norm_slots_that_name_nothing(sg):
    def edit(Z, R, slots, weights):
        slots[0] = -1                       # a token without experts
        slots[1, 1:] = -1
        slots[2, 0] = Z.shape[0]            # past the end
        slots[3, 2] = -(1 << 31)
        weights[1, 1:] = math.nan           # the weight of such a slot is not read
    check_norm(sg, 6, 264, k=3, edit=edit)


def test_norm_zero_rows(sg):
    def edit(Z, R, slots, weights):
        Z[0] = 0
        R[0] = 0
        Z[1] = 0
    Ro, H = check_norm(sg, 3, 64, eps=0.0, edit=edit)
    assert (Ro[0] == 0).all() and (H[0] == 0).all() and not torch.isnan(H).any()
    check_norm(sg, 3, 64, k=0, edit=edit)


@pytest.mark.parametrize("r32", [False, True])
def test_norm_in_place(sg, r32):
    check_norm(sg, 40, 896, k=2, r32=r32, inplace=True)


def test_norm_nan_stays_in_its_row(sg):
    Z = torch.randn(4, 64, generator=_gen("nn")).to(BF)
    Z[2, 5] = math.nan
    R = torch.randn(4, 64, generator=_gen("nr")).to(BF)
    Ro, H = sg.swiglu_residual_norm(Z.to(DEV), R.to(DEV))
    assert torch.isnan(H[2]).all() and not torch.isnan(H[[0, 1, 3]]).any() and not torch.isnan(Ro[[0, 1, 3]]).any()


@pytest.mark.parametrize("T", [9, 2000])
@pytest.mark.parametrize("post", [1, 0])
def test_norm_without_the_second_norm(sg, T, post):
    """H = NULL: only R' is made (the last block of a model)."""
    Z = torch.randn(T, 1024, generator=_gen("h0")).to(BF).to(DEV)
    R = torch.randn(T, 1024, generator=_gen("h1")).to(BF).to(DEV)
    want, _ = sg.swiglu_residual_norm(Z, R, post_norm=bool(post))
    out = torch.empty_like(R)
    rc = sg.lib().swiglu_residual_norm(Z.data_ptr(), None, None, R.data_ptr(), 0, post, None, None, 0, 1.0, None, 1e-6,
                                       out.data_ptr(), None, T, T, 0, 1024, torch.cuda.current_stream().cuda_stream)
    assert rc == sg.OK
    _status(sg)
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [0, 9, 2000])
@pytest.mark.parametrize("post", [True, False])
def test_norm_without_h_from_python(sg, T, post):
    """pre_norm=False: R' as with it, and no H."""
    gen = _gen("noh")
    Z, R = (torch.randn(T, 520, generator=gen).to(BF).to(DEV) for _ in range(2))
    gp = (1 + 0.2 * torch.randn(520, generator=gen)).to(BF).to(DEV) if post else None
    want, _ = sg.swiglu_residual_norm(Z, R, post_norm=post, gamma_post=gp, residual_scale=0.5)
    Ro, H = sg.swiglu_residual_norm(Z, R, post_norm=post, gamma_post=gp, residual_scale=0.5, pre_norm=False)
    _status(sg)
    assert H is None and torch.equal(Ro, want)
    Ro, H = sg.swiglu_residual_norm(Z, R, post_norm=post, gamma_post=gp, residual_scale=0.5, pre_norm=False, Rout=R)
    assert H is None and Ro is R and torch.equal(R, want)
    with pytest.raises(ValueError, match="gamma_pre without pre_norm"):
        sg.swiglu_residual_norm(Z, R, gamma_pre=want.new_ones(520), pre_norm=False)
    with pytest.raises(ValueError, match="H without pre_norm"):
        sg.swiglu_residual_norm(Z, R, H=torch.empty_like(Z), pre_norm=False)


def test_no_rows_and_no_choices(sg):
    # rows that name nothing at all, of a matrix with rows
    A = torch.ones(5, 16, dtype=BF, device=DEV)
    W = torch.ones(2, 16, 24, dtype=BF, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert sg.swiglu_linear_grouped(A, W, off, none).shape == (0, 24)
    assert sg.swiglu_fused_grouped(A, W, W, off, none).shape == (0, 24)
    # k = 0: nothing joins, R' = s R
    for T in (3, 900):
        R = torch.randn(T, 64, generator=_gen("k0")).to(BF).to(DEV)
        slots = torch.zeros(T, 0, dtype=torch.int32, device=DEV)
        Ro, _ = sg.swiglu_residual_norm(A.new_ones(7, 64), R, slots=slots, weights=torch.zeros(T, 0, device=DEV),
                                        residual_scale=0.5)
        _status(sg)
        assert torch.equal(Ro, (0.5 * R.float()).to(BF))


def test_norm_empty(sg):
    Z = torch.empty(0, 64, dtype=BF, device=DEV)
    Ro, H = sg.swiglu_residual_norm(Z, Z)
    assert Ro.shape == (0, 64) and H.shape == (0, 64)
    # tokens, but no expert rows at all
    R = torch.randn(3, 64, generator=_gen("e")).to(BF).to(DEV)
    slots = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    Ro, _ = sg.swiglu_residual_norm(Z, R, slots=slots, weights=torch.zeros(3, 2, device=DEV))
    assert torch.equal(Ro, R)


# ---- refusals of the binding -------------------------------------------------------


def test_binding_refusals(sg):
    x = torch.zeros(4, 16, dtype=BF, device=DEV)
    w = torch.zeros(2, 16, 24, dtype=BF, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="k must be"):
        sg.swiglu_moe_route(x, 17)
    with pytest.raises(ValueError, match="contiguous"):
        sg.swiglu_moe_route(x.t(), 2)
    with pytest.raises(ValueError, match="shape mismatch"):
        sg.swiglu_linear_grouped(torch.zeros(4, 8, dtype=BF, device=DEV), w, off)
    with pytest.raises(ValueError, match="offsets must have 3"):
        sg.swiglu_linear_grouped(x, w, off[:2])
    with pytest.raises(TypeError, match="int32"):
        sg.swiglu_linear_grouped(x, w, off.long())
    with pytest.raises(ValueError, match="W1 and W2"):
        sg.swiglu_fused_grouped(x, w, torch.zeros(3, 16, 24, dtype=BF, device=DEV), off)
    with pytest.raises(ValueError, match="the output"):
        sg.swiglu_linear_grouped(x, w, off, None, torch.empty(5, 24, dtype=BF, device=DEV))
    with pytest.raises(ValueError, match="go together"):
        sg.swiglu_residual_norm(x, x, slots=torch.zeros(4, 1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="gate must be"):
        sg.swiglu_residual_norm(x, x, gate=torch.zeros(5, 16, dtype=BF, device=DEV))
    with pytest.raises(ValueError, match="without post_norm"):
        sg.swiglu_residual_norm(x, x, gamma_post=x[0].contiguous(), post_norm=False)
    with pytest.raises(sg.SwigluError):
        sg.swiglu_residual_norm(x[:, :12].contiguous(), x[:, :12].contiguous())


# ---- the block ---------------------------------------------------------------------


def test_block_in_a_graph_matches_64_bits(sg):
    """Route, both products and the join, captured once and replayed on new
    inputs: the group sizes never leave the device."""
    T, Hd, F, E, k = 150, 264, 136, 12, 3
    gen = _gen("block")
    W1, W2 = [(torch.randn(E, Hd, F, generator=gen) / 16).to(BF) for _ in range(2)]
    W3 = (torch.randn(E, F, Hd, generator=gen) / 12).to(BF)
    x, lg, R = (torch.empty(T, n, dtype=BF, device=DEV) for n in (Hd, E, Hd))
    W1d, W2d, W3d = W1.to(DEV), W2.to(DEV), W3.to(DEV)
    state = {}

    def step():
        r = sg.swiglu_moe_route(lg, k, renormalize=True)
        y = sg.swiglu_fused_grouped(x, W1d, W2d, r.offsets, r.rows)
        z = sg.swiglu_linear_grouped(y, W3d, r.offsets)
        ro, h = sg.swiglu_residual_norm(z, R, slots=r.slots, weights=r.weights)
        state.update(r=r, y=y, z=z, ro=ro, h=h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.zero_(), lg.zero_(), R.zero_()
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        xs, ls, rs = (torch.randn(T, n, generator=gen).to(BF) for n in (Hd, E, Hd))
        ls[::7] = -math.inf
        x.copy_(xs), lg.copy_(ls), R.copy_(rs)
        graph.replay()
        _status(sg)
        r = state["r"]
        ids, w, offsets, rows, slots, _ = route_ref(ls.double().numpy(), k, True, 1.0)
        assert (r.ids.cpu().numpy() == ids).all() and (r.slots.cpu().numpy() == slots).all()
        n = offsets[-1]
        ref, tol = grouped_ref(xs, [W1, W2], offsets.tolist(), rows.tolist())
        assert ((state["y"].double().cpu() - ref).abs()[:n] <= tol[:n]).all()
        y = state["y"].cpu()
        ref, tol = grouped_ref(y, [W3], offsets.tolist(), None)
        assert ((state["z"].double().cpu() - ref).abs()[:n] <= tol[:n]).all()
        rr, hh, dr, dh = norm_ref(state["z"].cpu(), rs, torch.from_numpy(slots), r.weights.cpu(), True, None, None, 1.0,
                                  None, 1e-6)
        assert ((state["ro"].double().cpu() - rr).abs() <= dr + 2.0**-8 * rr.abs() + 1e-38).all()
        assert ((state["h"].double().cpu() - hh).abs() <= dh + 2.0**-8 * hh.abs() + 1e-38).all()


def test_example_block(sg):
    """The example's blocks against their plain form, and single tokens against the prompt.

    A block rounds Y and Z to BF16 (2^-9 each) and may round an element the
    other way than the plain form (2^-8 of it); as a norm over many elements
    such flips stay far below 2^-8.  Single tokens run the products in other
    tiles, with the sums in the same order over K: equal but for the router's
    logits, whose product may sum in another order and flip a rounding."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, off = mod.main(hidden=264, inner=136, experts=8, top_k=2, layers=2, prompt=81)
    assert worst < 2.0**-8 and off < 2.0**-6


# ---- sizes past 32 bits ---------------------------------------------------------------


def test_grouped_output_past_32_bits(sg):
    P, N, K = 70016, 32768, 64          # 2.3e9 outputs
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(P, K, generator=gen, device=DEV).to(BF)
    W = (torch.randn(2, K, N, generator=gen, device=DEV) / 8).to(BF)
    off = torch.tensor([0, 40000, P], dtype=torch.int32, device=DEV)
    Z = sg.swiglu_linear_grouped(X, W, off)
    _status(sg)
    for a, b, e in ((0, 3, 0), (39998, 40000, 0), (40000, 40002, 1), (65530, 65545, 1), (P - 3, P, 1)):
        ref, tol = grouped_ref(X[a:b].cpu(), [W[e:e + 1].cpu()], [0, b - a], None)
        assert ((Z[a:b].double().cpu() - ref).abs() <= tol).all(), (a, b)


def test_grouped_weights_past_32_bits(sg):
    E, K, N = 40, 2048, 28672           # 2.3e9 weights a matrix
    gen = torch.Generator(device="cuda").manual_seed(6)
    W = torch.empty(E, K, N, dtype=BF, device=DEV)
    for e in range(E):
        W[e] = torch.randn(K, N, generator=gen, device=DEV) / 45
    X = torch.randn(6, K, generator=gen, device=DEV).to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[36:] = 2
    off[38:] = 5
    off[40:] = 6
    Z = sg.swiglu_linear_grouped(X, W, off.to(DEV))
    _status(sg)
    for a, b, e in ((0, 2, 35), (2, 5, 37), (5, 6, 39)):
        ref, tol = grouped_ref(X[a:b].cpu(), [W[e:e + 1].cpu()], [0, b - a], None)
        assert ((Z[a:b].double().cpu() - ref).abs() <= tol).all(), e


def test_norm_past_32_bits(sg):
    T, D = 270000, 8192                 # 2.2e9 elements
    R = torch.zeros(T, D, dtype=BF, device=DEV)
    Z = torch.zeros(T, D, dtype=BF, device=DEV)
    at = [0, 1, 131071, 262143, 262144, T - 1]
    gen = torch.Generator(device="cuda").manual_seed(7)
    for t in at:
        R[t] = torch.randn(D, generator=gen, device=DEV)
        Z[t] = torch.randn(D, generator=gen, device=DEV)
    want = sg.swiglu_residual_norm(Z[at].contiguous(), R[at].contiguous())
    Ro, H = sg.swiglu_residual_norm(Z, R, Rout=R)
    _status(sg)
    assert torch.equal(Ro[at], want[0])
    assert ((H[at].float() - want[1].float()).abs() <= 2.0**-7 * want[1].float().abs()).all()
    assert int((H != 0).any(1).sum()) == len(at)
