"""GPU tests of the 8-bit quantisation and products against plain 64-bit
implementations (written here; no code shared with the library).

Tolerances, derived from the arithmetic:
  * quantisation: codes are exact; a scale is one FP32 quotient.
  * products: sums of products are whole numbers, exact below 2^24; a sum whose
    terms' magnitudes S pass that is off by at most K 2^-23 S (truncating FP32
    additions included).  Conversion and scales: three FP32 roundings; the
    result's rounding to BF16 is half a step, 2^-8 relative.  For SiLU(g) u the
    errors of g and u enter with |d SiLU| <= 1.1, fast exp and divide with 2^-19.
"""
import math
import zlib

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, I8, F32 = torch.bfloat16, torch.int8, torch.float32


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


# ---- quantisation ---------------------------------------------------------------


def quant_ref(X):
    x = X.double()
    top = x.abs().amax(-1, keepdim=True) if x.shape[-1] else x.new_zeros(*x.shape[:-1], 1)
    q = torch.round(127 * x / top)  # halves to even
    q = torch.where((top > 0) & torch.isfinite(top), q, 0.0)
    scale = torch.where(torch.isfinite(top), (top.float() / 127), math.nan)
    return q.to(I8), scale.squeeze(-1).float()


def check_quant(sg, X, **kw):
    q, s = sg.swiglu_quant_int8(X.to(DEV), **kw)
    assert q.dtype == I8 and s.dtype == F32 and q.shape == X.shape and s.shape == X.shape[:-1]
    want, scale = quant_ref(X)
    assert torch.equal(q.cpu(), want)
    assert torch.equal(torch.nan_to_num(s.cpu(), nan=-1.0), torch.nan_to_num(scale, nan=-1.0))
    return q, s


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 8), (9, 16), (61, 1024), (33, 1032), (5, 4096), (17, 4104), (3, 8192), (2, 8200), (3, 32768),
                                   (2, 32776), (1, 100000), (3, 7, 264), (2, 300, 896), (2000, 128)], ids=lambda s: "x".join(map(str, s)))
def test_quant(sg, shape, dtype):
    check_quant(sg, (torch.randn(*shape, generator=_gen("quant", shape)) * 3).to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_quant_halves_go_to_even(sg, dtype):
    x = torch.arange(-127, 128).float().repeat(4)[:1016].unsqueeze(0)  # max 127 * 2^p: halves below
    rows = [x * 2.0, torch.cat([x * 0.5 + 0.25, torch.full((1, 8), 127.0)], 1)[:, :1016]]
    top = torch.arange(1, 256).float()
    many = torch.cat([top[:, None], torch.arange(0, 255).float().expand(255, 255) * top[:, None] / 254], 1)  # odd 254ths of each max
    check_quant(sg, torch.cat(rows).to(dtype))
    check_quant(sg, many[:, :256].contiguous().to(dtype))
    # one FP32 step to either side of a half
    if dtype == F32:
        h = (torch.arange(0, 127).float() + 0.5) / 127
        up, down = torch.nextafter(h, h + 1), torch.nextafter(h, h - 1)
        check_quant(sg, torch.cat([h, up, down, -h, -up, -down, torch.ones(6)])[None, :768].contiguous())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K", [64, 40000])
def test_quant_rows_out_of_the_ordinary(sg, dtype, K):
    x = torch.randn(12, K, generator=_gen("odd", K))
    x[0] = 0.0
    x[1, 5] = math.nan
    x[2, K - 1] = -math.inf
    x[3] *= 1e-40      # subnormal
    x[4] *= 1e37
    x[5] = -0.0
    x[6] = 0.0
    x[6, 3] = torch.finfo(dtype).smallest_normal
    x[7] = torch.finfo(dtype).max
    x[8, 1:] = 0.0
    x[9, 7] = 1e30     # one value above all others
    check_quant(sg, x.to(dtype))


def test_quant_empty(sg):
    q, s = sg.swiglu_quant_int8(torch.empty(0, 16, device=DEV))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = sg.swiglu_quant_int8(torch.empty(5, 0, device=DEV, dtype=BF))
    assert s.tolist() == [0.0] * 5


def test_quant_into_given_outputs_and_refusals(sg):
    x = torch.randn(6, 32, generator=_gen("given")).to(DEV)
    Q, S = torch.empty(6, 32, dtype=I8, device=DEV), torch.empty(6, device=DEV)
    q, s = sg.swiglu_quant_int8(x, Q, S)
    assert q.data_ptr() == Q.data_ptr() and s.data_ptr() == S.data_ptr()
    assert torch.equal(Q.cpu(), quant_ref(x.cpu())[0])
    for bad in (x[0], x.t(), x[:, ::2], x[None, None]):
        with pytest.raises(ValueError):
            sg.swiglu_quant_int8(bad)
    with pytest.raises(ValueError):
        sg.swiglu_quant_int8(x, Q[:5])
    with pytest.raises(TypeError):
        sg.swiglu_quant_int8(x, Q.float())
    with pytest.raises(sg.SwigluError):
        sg.swiglu_quant_int8(x[:, :28].contiguous())


# ---- products ---------------------------------------------------------------------


def product_ref(A, sa, Ws, offsets, rows):
    """(value, allowed error) in 64 bits; NaN where no expert owns the place."""
    A, sa = A.to(DEV).double(), sa.to(DEV).double()
    P = len(rows) if rows is not None else A.shape[0]
    N, K = Ws[0][0].shape[1:]
    ref = torch.full((P, N), math.nan, dtype=torch.double, device=DEV)
    tol = torch.zeros_like(ref)
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a >= b:
            continue
        if rows is None:
            x, s, ok = A[a:b], sa[a:b], torch.ones(b - a, dtype=torch.bool, device=DEV)
        else:
            r = torch.tensor(rows[a:b], device=DEV)
            ok = (r >= 0) & (r < A.shape[0])
            r = r.clamp(0, A.shape[0] - 1)
            x, s = A[r], sa[r]
        out = []
        for W, w in Ws:
            wd, scale = W[e].to(DEV).double(), s[:, None] * w[e].to(DEV).double()
            size = x.abs() @ wd.abs().t()
            z = (x @ wd.t()) * scale
            out.append((z, torch.where(size >= 2.0**24, K * 2.0**-23 * size, 0.0) * scale.abs() + 3 * 2.0**-24 * z.abs()))
        (g, dg), (u, du) = out[0], out[-1]
        if len(Ws) == 1:
            y, t = g, dg
        else:
            h = g * torch.sigmoid(g)
            y, t = h * u, 1.1 * dg * (u.abs() + du) + h.abs() * du + 2.0**-19 * (h * u).abs()
        ref[a:b], tol[a:b] = torch.where(ok[:, None], y, 0.0), torch.where(ok[:, None], t, 0.0)
    return ref, tol + 2.0**-8 * ref.abs() + 1e-37


SENTINEL = -77.0


def check_product(sg, fused, sizes, N, K, T=None, first=0, spare=0, seed=0, edit=None, dense=False, full=False):
    """sizes: rows of each expert; T: rows of A that `rows` draws from (None: no rows); full: codes of one sign, the largest."""
    E = len(sizes)
    gen = _gen("int8", fused, tuple(sizes), N, K, seed)
    offsets = [first]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    P = offsets[-1] + spare
    codes = (lambda *s: torch.randint(-128, -126, s, generator=gen).to(I8)) if full else (lambda *s: torch.randint(-128, 128, s, generator=gen).to(I8))
    M = P if T is None else T
    A, sa = codes(M, K), torch.rand(M, generator=gen) * 0.02 + 1e-3
    Ws = [(codes(E, N, K), (torch.rand(E, N, generator=gen) + 0.1) * 0.02 / math.sqrt(max(K, 1)) * (0.1 if full else 1)) for _ in range(2 if fused else 1)]
    rows = None if T is None else torch.randint(0, T, (P,), generator=gen).tolist()
    if edit:
        edit(A, sa, Ws, rows)
    Y = torch.full((P, N), SENTINEL, dtype=BF, device=DEV)
    args = [A.to(DEV), sa.to(DEV)]
    for W, w in Ws:
        args += [W.to(DEV)[0], w.to(DEV)[0]] if dense else [W.to(DEV), w.to(DEV)]
    if dense:
        (sg.swiglu_fused_int8 if fused else sg.swiglu_linear_int8)(*args, Y)
    else:
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        rd = None if rows is None else torch.tensor(rows, dtype=torch.int32, device=DEV)
        (sg.swiglu_fused_grouped_int8 if fused else sg.swiglu_linear_grouped_int8)(*args, off, rd, Y)
    _status(sg)
    ref, tol = product_ref(A, sa, Ws, offsets, rows)
    got = Y.double()
    assert (got[:first] == SENTINEL).all() and (got[offsets[-1]:] == SENTINEL).all()
    body = slice(first, offsets[-1])
    want_nan = torch.isnan(ref[body])
    assert torch.equal(torch.isnan(got[body]), want_nan)
    err = torch.where(want_nan, 0.0, (got - ref).abs()[body])
    bad = err > torch.where(want_nan, 1.0, tol[body])
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}, worst {(err / tol[body]).max()}"
    return Y


FORMS = pytest.mark.parametrize("fused", [True, False], ids=["fused", "linear"])


@FORMS
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 100, 128, 129, 191, 192, 193, 257, 700])
@pytest.mark.parametrize("NK", [(8, 16), (72, 144), (264, 208), (520, 1104), (128, 4880)], ids=lambda s: "x".join(map(str, s)))
def test_dense(sg, fused, M, NK):
    check_product(sg, fused, [M], *NK, dense=True)


@FORMS
@pytest.mark.parametrize("gather", [True, False], ids=["rows", "dense"])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [0, 0, 1, 0], [31, 32, 33], [64, 65, 1, 0, 63], [191, 192, 193, 0, 2],
                                   [700, 0, 0, 1, 513], [95, 96, 97, 385]], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("NK", [(8, 16), (72, 144), (264, 208), (512, 64)], ids=lambda s: "x".join(map(str, s)))
def test_grouped(sg, fused, gather, sizes, NK):
    check_product(sg, fused, sizes, *NK, T=53 if gather else None)


@FORMS
@pytest.mark.parametrize("gather", [True, False], ids=["rows", "dense"])
@pytest.mark.parametrize("sizes", [[33, 0], [0, 20, 0, 1], [5, 33, 0, 70], [128, 1], [300], [17, 0, 0, 0, 0, 0, 0, 0, 0, 1]],
                         ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("NK", [(8, 1024), (72, 1040), (264, 1104), (520, 2064), (2600, 1120)], ids=lambda s: "x".join(map(str, s)))
def test_grouped_few_units_share_k(sg, fused, gather, sizes, NK):
    check_product(sg, fused, sizes, *NK, T=11 if gather else None)


@FORMS
@pytest.mark.parametrize("E,rows_each,N,K", [(1024, 3, 1024, 32), (16, 1300, 4096, 48)], ids=["short", "long"])
def test_grouped_ring_of_units_wraps(sg, fused, E, rows_each, N, K):
    check_product(sg, fused, [rows_each + (e % 3) for e in range(E)], N, K, T=100)


@FORMS
@pytest.mark.parametrize("E", [8, 64])
@pytest.mark.parametrize("P", [15, 16, 17, 31, 32, 33, 64, 65])
def test_grouped_few_places_of_large_matrices(sg, fused, E, P):
    sizes = torch.bincount(torch.randint(0, E, (P,), generator=_gen("places", E, P)), minlength=E).tolist()
    check_product(sg, fused, sizes, 1368, 3008, T=P // 2 + 1)


@FORMS
@pytest.mark.parametrize("E", [1, 2, 31, 32, 33, 64, 257, 1024])
def test_grouped_expert_counts(sg, fused, E):
    sizes = torch.randint(0, 4, (E,), generator=_gen("experts", E)).tolist()
    sizes[-1] = 1
    check_product(sg, fused, sizes, 40, 48, T=17)


@FORMS
def test_one_token(sg, fused):
    check_product(sg, fused, [0, 1, 0, 0, 1, 1, 0, 1], 1024, 2048, T=1)
    check_product(sg, fused, [1], 2568, 3584, dense=True)


@FORMS
def test_more_units_than_pairs(sg, fused):
    check_product(sg, fused, [300, 17, 0, 520, 64, 1, 129, 33], 2568, 144, T=200)
    check_product(sg, fused, [1500], 4872, 272, dense=True)


@FORMS
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("sizes", [[3, 0, 40], [1, 0, 1]])
def test_grouped_leaves_other_places_alone(sg, fused, gather, sizes):
    check_product(sg, fused, sizes, 136, 80, T=9 if gather else None, first=5, spare=11)


@FORMS
@pytest.mark.parametrize("M", [3, 300])
def test_sums_past_24_bits(sg, fused, M):
    # every product near 2^14: sums of 2^27
    check_product(sg, fused, [M], 136, 9216, dense=True, full=True)


@pytest.mark.parametrize("M", [1, 2, 40, 200])
def test_sums_are_exact_up_to_24_bits(sg, M):
    """K = 1024 products of 127 or 128 squared, told apart by one: scales of one make Z the rounded integer."""
    K, N = 1024, 64
    A = torch.full((M, K), -128, dtype=I8)
    W = torch.full((N, K), -128, dtype=I8)
    W[:, 0] = torch.arange(N) - 128
    A[:, 1:3] = torch.randint(-128, 127, (M, 2), generator=_gen("exact")).to(I8)
    W[:, 3:] *= torch.tensor([1, 0], dtype=I8).repeat(511)[:1021]  # stay inside 2^24
    one = torch.ones(max(M, N), device=DEV)
    Z = sg.swiglu_linear_int8(A.to(DEV), one[:M].contiguous(), W.to(DEV), one[:N].contiguous())
    want = (A.long() @ W.long().t()).float().to(BF)
    assert torch.equal(Z.cpu(), want)
    # the low bits decide as well: subtract a multiple of 256 by products of the other sign
    W2 = torch.cat([W, W.neg().clamp(-127)], 1)
    A2 = torch.cat([A, A], 1)
    Z = sg.swiglu_linear_int8(A2.to(DEV), one[:M].contiguous(), W2.to(DEV), one[:N].contiguous())
    assert torch.equal(Z.cpu(), (A2.long() @ W2.long().t()).float().to(BF))


@pytest.mark.parametrize("M", [1, 40, 200])
def test_long_k(sg, M):
    # past 2^17 an FP32 or a 32-bit sum of the largest products would pass its range
    check_product(sg, False, [M], 16, (1 << 17) + 48, dense=True, full=True)


@FORMS
@pytest.mark.parametrize("T", [6, 200])
def test_row_numbers_outside_a_give_zeros(sg, fused, T):
    def edit(A, sa, Ws, rows):
        for i, r in enumerate((-1, T, -(1 << 31), (1 << 31) - 1)):
            rows[3 * i + 1] = r
        sa[0] = math.nan  # (the clamped row's scale does not reach them)
        for i in range(len(rows)):
            rows[i] = 1 if rows[i] == 0 else rows[i]
    Y = check_product(sg, fused, [13, 2] if T == 6 else [130, 70], 72, 144, T=T, edit=edit)
    assert (Y[1] == 0).all() and (Y[4] == 0).all() and (Y[7] == 0).all()


@FORMS
@pytest.mark.parametrize("M", [4, 150])
def test_scales_that_are_nan_or_zero_stay_in_their_row_and_column(sg, fused, M):
    def edit(A, sa, Ws, rows):
        sa[1], sa[2] = math.nan, 0.0
        Ws[0][1][0, 5] = math.nan
        Ws[-1][1][0, 6] = 0.0
    check_product(sg, fused, [M], 72, 144, dense=True, edit=edit)


@FORMS
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("offsets", [[0, 30, 10, 50], [-5, 10, 20, 90], [40, 30, 20, 10], [60, 60, 60, 60]])
def test_malformed_offsets_stay_in_bounds(sg, fused, few, offsets):
    """Clamped to [0, P] and made not decreasing."""
    P = 3 if few else 60
    offsets = [min(o, 3) for o in offsets] if few else offsets
    gen = _gen("malformed")
    q = lambda *s: torch.randint(-127, 128, s, generator=gen).to(I8).to(DEV)  # noqa: E731
    f = lambda *s: (torch.rand(*s, generator=gen) * 0.01).to(DEV)  # noqa: E731
    A, sa = q(P, 64), f(P)
    Ws = [q(3, 40, 64), f(3, 40)] * (2 if fused else 1)
    fn = sg.swiglu_fused_grouped_int8 if fused else sg.swiglu_linear_grouped_int8
    Y = [torch.full((P, 40), SENTINEL, dtype=BF, device=DEV) for _ in range(2)]
    fn(A, sa, *Ws, torch.tensor(offsets, dtype=torch.int32, device=DEV), None, Y[0])
    clean, top = [], 0
    for o in offsets:
        top = max(top, min(max(o, 0), P))
        clean.append(top)
    fn(A, sa, *Ws, torch.tensor(clean, dtype=torch.int32, device=DEV), None, Y[1])
    _status(sg)
    assert torch.equal(Y[0], Y[1])


@FORMS
def test_zero_k_and_no_rows(sg, fused):
    z = lambda *s, d=I8: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    fn = sg.swiglu_fused_grouped_int8 if fused else sg.swiglu_linear_grouped_int8
    n = 2 if fused else 1
    Y = torch.full((5, 16), SENTINEL, dtype=BF, device=DEV)
    fn(z(5, 0), z(5, d=F32), *[z(2, 16, 0), z(2, 16, d=F32)] * n, off, None, Y)
    assert (Y == 0).all()
    Y.fill_(SENTINEL)
    fn(z(0, 32), z(0, d=F32), *[z(2, 16, 32), z(2, 16, d=F32)] * n, off, z(5, d=torch.int32), Y)
    assert (Y == 0).all()
    assert fn(z(4, 32), z(4, d=F32), *[z(2, 16, 32), z(2, 16, d=F32)] * n, off, z(0, d=torch.int32)).shape == (0, 16)
    dense = sg.swiglu_fused_int8 if fused else sg.swiglu_linear_int8
    assert dense(z(0, 32), z(0, d=F32), *[z(16, 32), z(16, d=F32)] * n).shape == (0, 16)
    assert dense(z(4, 32), z(4, d=F32), *[z(0, 32), z(0, d=F32)] * n).shape == (4, 0)
    assert (dense(z(4, 0), z(4, d=F32), *[z(16, 0), z(16, d=F32)] * n) == 0).all()


@FORMS
@pytest.mark.parametrize("sizes", [[1, 0, 2], [40, 0, 5], [300, 200, 7]])
def test_repeats_bit_for_bit_on_another_stream(sg, fused, sizes):
    a = check_product(sg, fused, sizes, 264, 1104, T=50)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = check_product(sg, fused, sizes, 264, 1104, T=50)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_binding_refusals(sg):
    q, s = torch.zeros(4, 32, dtype=I8, device=DEV), torch.zeros(4, device=DEV)
    W, w = torch.zeros(16, 32, dtype=I8, device=DEV), torch.zeros(16, device=DEV)
    We, we = W[None].repeat(3, 1, 1), w[None].repeat(3, 1)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    for call, err in ((lambda: sg.swiglu_linear_int8(q.to(torch.uint8), s, W, w), TypeError),
                      (lambda: sg.swiglu_linear_int8(q, s.to(BF), W, w), TypeError),
                      (lambda: sg.swiglu_linear_int8(q, s[:3], W, w), ValueError),
                      (lambda: sg.swiglu_linear_int8(q, s, W, w[:8]), ValueError),
                      (lambda: sg.swiglu_linear_int8(q, s, W[:, :16].contiguous(), w), ValueError),
                      (lambda: sg.swiglu_linear_int8(q, s, W.t(), w), ValueError),
                      (lambda: sg.swiglu_fused_int8(q, s, W, w, W[:8], w[:8]), ValueError),
                      (lambda: sg.swiglu_fused_int8(q, s, W, w, W, None), TypeError),
                      (lambda: sg.swiglu_linear_int8(q, s, W, w, torch.zeros(4, 8, dtype=BF, device=DEV)), ValueError),
                      (lambda: sg.swiglu_linear_grouped_int8(q, s, We, we, off[:3]), ValueError),
                      (lambda: sg.swiglu_linear_grouped_int8(q, s, We, w, off), ValueError),
                      (lambda: sg.swiglu_linear_grouped_int8(q, s, We, we, off.long()), TypeError),
                      (lambda: sg.swiglu_linear_grouped_int8(q, s, W, w, off), ValueError),
                      (lambda: sg.swiglu_linear_int8(q[:, :24].contiguous(), s, W[:, :24].contiguous(), w), sg.SwigluError)):
        with pytest.raises(err):
            call()
    _status(sg)


def test_the_longest_k_of_the_largest_codes(sg):
    K = (1 << 20) - 1024
    A, W = torch.full((8, K), -128, dtype=I8, device=DEV), torch.full((16, K), -128, dtype=I8, device=DEV)
    a, w = torch.full((8,), 2.0**-20, device=DEV), torch.full((16,), 2.0**-14, device=DEV)
    for M in (1, 8):
        assert (sg.swiglu_linear_int8(A[:M], a[:M], W, w).float() == torch.tensor(K * 2.0**-20).to(BF).float()).all()
    with pytest.raises(sg.SwigluError):
        sg.swiglu_linear_int8(torch.zeros(1, K + 16, dtype=I8, device=DEV), a[:1], torch.zeros(16, K + 16, dtype=I8, device=DEV), w)


def test_rows_alone_and_together_give_the_same_bits(sg):
    """A row's result does not depend on how many rows the call has (sums below 2^24 are exact in every form)."""
    gen = _gen("alone")
    q = lambda *s: torch.randint(-127, 128, s, generator=gen).to(I8).to(DEV)  # noqa: E731
    A, a = q(400, 1024), (torch.rand(400, generator=gen) * 0.01).to(DEV)
    W1, W2 = ((q(520, 1024), (torch.rand(520, generator=gen) * 0.01).to(DEV)) for _ in range(2))
    for fn, ws in ((sg.swiglu_fused_int8, (*W1, *W2)), (sg.swiglu_linear_int8, W1)):
        whole = fn(A, a, *ws)
        for m in (1, 7, 30, 150):
            assert torch.equal(fn(A[:m], a[:m], *ws), whole[:m])


@pytest.mark.parametrize("K", [16, 48])
def test_output_past_32_bits(sg, K):
    P, N = 70016, 32768          # 2.3e9 outputs
    gen = torch.Generator(device="cuda").manual_seed(5)
    A = torch.randint(-127, 128, (P, K), generator=gen, device=DEV).to(I8)
    W = torch.randint(-127, 128, (2, N, K), generator=gen, device=DEV).to(I8)
    a, w = torch.rand(P, generator=gen, device=DEV) * 0.01, torch.rand(2, N, generator=gen, device=DEV) * 0.01
    off = torch.tensor([0, 40000, P], dtype=torch.int32, device=DEV)
    Z = sg.swiglu_linear_grouped_int8(A, a, W, w, off)
    _status(sg)
    for i, j, e in ((0, 3, 0), (39998, 40000, 0), (40000, 40002, 1), (65530, 65545, 1), (P - 3, P, 1)):
        ref, tol = product_ref(A[i:j], a[i:j], [(W[e:e + 1], w[e:e + 1])], [0, j - i], None)
        assert ((Z[i:j].double() - ref).abs() <= tol).all(), (i, j)


@pytest.mark.parametrize("P", [6, 70, 3000])
def test_weights_past_32_bits(sg, P):
    E, N, K = 40, 28672, 2048    # 2.3e9 weights
    gen = torch.Generator(device="cuda").manual_seed(6)
    W, w = torch.empty(E, N, K, dtype=I8, device=DEV), torch.rand(E, N, generator=gen, device=DEV) * 1e-3
    for e in range(E):
        W[e] = torch.randint(-127, 128, (N, K), generator=gen, device=DEV)
    A, a = torch.randint(-127, 128, (P, K), generator=gen, device=DEV).to(I8), torch.rand(P, generator=gen, device=DEV) * 0.01
    cut = [0, P // 3, P // 3 + 3 * P // 6, P]
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[36:], off[38:], off[40:] = cut[1], cut[2], cut[3]
    Z = sg.swiglu_linear_grouped_int8(A, a, W, w, off.to(DEV))
    _status(sg)
    for i, e in zip(range(3), (35, 37, 39)):
        x, y = cut[i], min(cut[i + 1], cut[i] + 40)
        ref, tol = product_ref(A[x:y], a[x:y], [(W[e:e + 1], w[e:e + 1])], [0, y - x], None)
        assert ((Z[x:y].double() - ref).abs() <= tol).all(), e


def test_rows_past_32_bits(sg):
    T, K = 70016, 32768          # 2.3e9 codes, quantised and multiplied
    X = torch.zeros(T, K, dtype=BF, device=DEV)
    at = [0, 1, 65534, 65535, 65536, 65537, T - 1]
    gen = torch.Generator(device="cuda").manual_seed(7)
    for t in at:
        X[t] = torch.randn(K, generator=gen, device=DEV)
    q, s = sg.swiglu_quant_int8(X)
    want, scale = quant_ref(X[at].cpu())
    assert torch.equal(q[at].cpu(), want) and torch.equal(s[at].cpu(), scale)
    assert int((q != 0).any(1).sum()) == len(at)
    del X
    W, w = torch.randint(-127, 128, (72, K), generator=gen, device=DEV).to(I8), torch.rand(72, generator=gen, device=DEV) * 1e-3
    Z = sg.swiglu_linear_int8(q, s, W, w)
    _status(sg)
    ref, tol = product_ref(q[at], s[at], [(W[None], w[None])], [0, len(at)], None)
    assert ((Z[at].double() - ref).abs() <= tol).all()
    assert int((Z != 0).any(1).sum()) == len(at)


# ---- the calls together -----------------------------------------------------------


@pytest.fixture(scope="module")
def block(sg):
    from examples import moe_block_int8
    return moe_block_int8.SparseBlockInt8(272, 144, 16, 4, seed=3)


def check_stages(block, R, H, stages, out):
    """Every stage against the 64-bit form of its own inputs."""
    route = stages["route"]
    for x, q in ((H, stages["Hq"]), (stages["Y"], stages["Yq"])):
        want, scale = quant_ref(x.cpu())
        assert torch.equal(q[0].cpu(), want) and torch.equal(q[1].cpu(), scale)
    offsets, rows = route.offsets.tolist(), route.rows.tolist()
    assert sorted(rows) == sorted(list(range(R.shape[0])) * block.top_k) and offsets[-1] == len(rows)
    for a, Ws, r, got in ((stages["Hq"], [block.Q1, block.Q2], rows, stages["Y"]), (stages["Yq"], [block.Q3], None, stages["Z"])):
        ref, tol = product_ref(*a, Ws, offsets, r)
        assert ((got.double() - ref).abs() <= tol).all()
    # the norms: 128 roundings of 2^-24 of the terms' magnitudes, and one to BF16
    w, z = route.weights.double(), stages["Z"].double()[route.slots.long()]
    joined, size = (w[..., None] * z).sum(1), (w[..., None] * z).abs().sum(1)
    gate = block.gate.double()
    rms = torch.sqrt(joined.square().mean(1, keepdim=True) + block.eps)
    r = R.double() + gate * joined / rms
    tol = 128 * 2.0**-24 * (R.double().abs() + gate * (size + joined.abs()) / rms)
    assert ((out[0].double() - r).abs() <= tol).all()
    h = r / torch.sqrt(r.square().mean(1, keepdim=True) + block.eps)
    assert ((out[1].double() - h).abs() <= 2.0**-8 * h.abs() + 4 * tol + 1e-30).all()


@pytest.mark.parametrize("T", [1, 5, 300])
def test_block_in_a_graph_replayed_on_new_inputs(sg, block, T):
    R, H, stages = torch.zeros(T, 272, device=DEV), torch.zeros(T, 272, dtype=BF, device=DEV), {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(R, H)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(R, H, stages)
    for i in range(3):
        gen = _gen("block", T, i)
        R.copy_(torch.randn(T, 272, generator=gen))
        H.copy_(torch.randn(T, 272, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        _status(sg)
        check_stages(block, R, H, stages, out)


def test_two_graphs_and_an_eager_call_in_turn(sg, block):
    """Graphs captured one after the other, replayed in turn: each has workspaces of its own."""
    ins = [(torch.randn(T, 272, generator=_gen("two", T)).to(DEV), torch.randn(T, 272, generator=_gen("2", T)).to(DEV, BF)) for T in (300, 180)]
    want = [[t.clone() for t in block(*x)] for x in ins]
    graphs = []
    for x in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, block(*x)))
    for _ in range(3):
        for (g, out), w in zip(graphs, want):
            for t in out:
                t.zero_()
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
        assert all(torch.equal(a, b) for a, b in zip(block(*ins[0]), want[0]))
    _status(sg)


@pytest.mark.parametrize("stream", [lambda s: s, lambda s: s.cuda_stream], ids=["object", "handle"])
def test_outputs_and_workspaces_belong_to_the_stream_of_the_call(sg, stream):
    """Memory that the current stream has queued work for is not handed to a call
    on another stream, nor the call's workspace to the current stream."""
    T, E, k, N, K = 4096, 64, 8, 256, 128
    s = torch.cuda.Stream()
    gen = _gen("pools")
    lg, x = torch.randn(T, E, generator=gen).to(DEV), torch.randn(T, K, generator=gen).to(DEV, BF)
    W1, W2, W3 = (sg.swiglu_quant_int8(torch.randn(E, n, m, generator=gen).to(DEV)) for n, m in ((N, K), (N, K), (K, N)))
    D = sg.swiglu_quant_int8(torch.randn(N, K, generator=gen).to(DEV))

    def step(**kw):
        r = sg.swiglu_moe_route_scored(lg, k, groups=8, kept_groups=4, **kw)
        q = sg.swiglu_quant_int8(x, **kw)
        y = sg.swiglu_fused_grouped_int8(*q, *W1, *W2, r.offsets, r.rows, **kw)
        yq = sg.swiglu_quant_int8(y, **kw)
        z = sg.swiglu_linear_grouped_int8(*yq, *W3, r.offsets, **kw)
        return [*r, *q, y, *yq, z, sg.swiglu_linear_int8(*q, *D, **kw), sg.swiglu_fused_int8(*q, *D, *D, **kw)]

    want = [t.cpu() for t in step()]
    sizes = [t.numel() * t.element_size() for t in want] + [T * K * 2, T * k * N * 2]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x7F)
    got = step(stream=stream(s))
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    late = step(stream=stream(s))
    for n in sizes * 2:
        torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x7F)
    torch.cuda.synchronize()
    _status(sg)
    for w, a, b in zip(want, got, late):
        assert torch.equal(w, a.cpu()) and torch.equal(w, b.cpu())


@pytest.mark.parametrize("M", [1, 8, 33, 125, 700])
def test_calls_wait_for_the_makers_of_all_their_operands(sg, M):
    """Codes and scales of rows and weights made anew, in the same buffers, right before each
    product; a large product in front keeps the GPU busy while all are launched."""
    K, N, turns = 4864, 896, 6
    g = _gen("chain", M)
    Xs = [torch.randn(M, K, generator=g).to(BF).to(DEV) for _ in range(turns)]
    Ws = [torch.randn(N, K, generator=g).to(BF).to(DEV) for _ in range(turns)]
    big, bs = sg.swiglu_quant_int8(torch.randn(4096, K, generator=g).to(BF).to(DEV))
    A, sa = sg.swiglu_quant_int8(Xs[0])
    W, sw = sg.swiglu_quant_int8(Ws[0])
    want = []
    for X, V in zip(Xs, Ws):
        one = (*sg.swiglu_quant_int8(X), *sg.swiglu_quant_int8(V))
        torch.cuda.synchronize()
        want.append(sg.swiglu_linear_int8(*one))
        torch.cuda.synchronize()
    Y = torch.zeros(M, N, dtype=BF, device=DEV)
    got = []
    sg.swiglu_linear_int8(big, bs, big, bs)
    for X, V in zip(Xs, Ws):
        sg.swiglu_quant_int8(X, A, sa)
        sg.swiglu_quant_int8(V, W, sw)
        got.append(sg.swiglu_linear_int8(A, sa, W, sw, Y).clone())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_given_workspaces_and_their_refusals(sg):
    gen = _gen("workspace")
    q = lambda *s: torch.randint(-127, 128, s, generator=gen).to(I8).to(DEV)  # noqa: E731
    A, a, W, w = q(700, 256), torch.rand(700, generator=gen).to(DEV), q(512, 256), torch.rand(512, generator=gen).to(DEV)
    need = sg.lib().swiglu_int8_workspace_size(700, 700, 0, 512, 256, 0)
    assert need == 700 * 256 * 2
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert torch.equal(sg.swiglu_linear_int8(A, a, W, w, workspace=ws), sg.swiglu_linear_int8(A, a, W, w))
    for bad in (ws[:-1], ws[8:], ws[:0]):
        with pytest.raises(sg.SwigluError):
            sg.swiglu_linear_int8(A, a, W, w, workspace=bad)
    _status(sg)


def test_example_block(sg):
    from examples import moe_block_int8
    worst, off = moe_block_int8.main(hidden=272, inner=144, experts=16, top_k=4, layers=2, prompt=90)
    # BF16 roundings of Y and Z that fall the other way, a few in a thousand
    assert worst < 2.0**-8 and off < 2.0**-8


@pytest.mark.parametrize("M", [1, 8, 33, 125, 700])
def test_operands_made_anew_in_an_unbroken_chain(sg, M):
    """As test_calls_wait_for_the_makers_of_all_their_operands, each turn with an output of its own, so
    that no ordinary launch parts the turns: several of these kernels are resident together."""
    K, N, turns = 4864, 896, 6
    g = _gen("unbroken", M)
    Xs = [torch.randn(M, K, generator=g).to(BF).to(DEV) for _ in range(turns)]
    Ws = [torch.randn(N, K, generator=g).to(BF).to(DEV) for _ in range(turns)]
    want = []
    for X, V in zip(Xs, Ws):
        one = (*sg.swiglu_quant_int8(X), *sg.swiglu_quant_int8(V))
        torch.cuda.synchronize()
        want.append(sg.swiglu_fused_int8(*one, *one[2:]))
        torch.cuda.synchronize()
    A, sa = sg.swiglu_quant_int8(Xs[0])
    W, sw = sg.swiglu_quant_int8(Ws[0])
    ws = torch.empty(max(sg.lib().swiglu_int8_workspace_size(M, M, 0, N, K, 1), 16), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = [torch.zeros(M, N, dtype=BF, device=DEV) for _ in range(turns)]
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)
        for X, V, Y in zip(Xs, Ws, got):
            sg.swiglu_quant_int8(X, A, sa)
            sg.swiglu_quant_int8(V, W, sw)
            sg.swiglu_fused_int8(A, sa, W, sw, W, sw, Y, workspace=ws)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    _status(sg)


@pytest.mark.parametrize("T", [1, 5, 40, 300, 700])
def test_a_block_of_buffers_used_again_in_an_unbroken_chain(sg, T):
    """Routing, codes, offsets, rows and outputs written anew in the same buffers turn by turn,
    by kernels that are resident together; only the last norm's outputs are a turn's own."""
    E, k, N, K, turns = 32, 4, 256, 384, 6
    g = _gen("unbroken block", T)
    W1, W2, W3 = (sg.swiglu_quant_int8(torch.randn(E, n, m, generator=g).to(DEV)) for n, m in ((N, K), (N, K), (K, N)))
    bias = (torch.randn(E, generator=g) * 0.1).to(DEV)
    ins = [(torch.randn(T, E, generator=g).to(DEV), torch.randn(T, K, generator=g).to(BF).to(DEV), torch.randn(T, K, generator=g).to(DEV))
           for _ in range(turns)]
    size = sg.lib().swiglu_int8_workspace_size
    e = lambda *s, d=F32: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731

    def buffers():
        P = T * k
        return dict(ids=e(T, k, d=torch.int32), weights=e(T, k), offsets=e(E + 1, d=torch.int32), rows=e(P, d=torch.int32),
                    slots=e(T, k, d=torch.int32), workspace=e(max(sg.lib().swiglu_moe_route_workspace_size(T, E, k), 16), d=torch.uint8)), dict(
                    A=e(T, K, d=I8), a=e(T), Y=e(P, N, d=BF), B=e(P, N, d=I8), b=e(P), Z=e(P, K, d=BF),
                    ws=e(max(size(T, P, E, N, K, 1), size(P, P, E, K, N, 0), 16), d=torch.uint8))

    def turn(x, route, m, out, pause):
        logits, H, R = x
        sg.swiglu_moe_route_scored(logits, k, bias=bias, groups=4, kept_groups=2, **route)
        pause()
        sg.swiglu_quant_int8(H, m["A"], m["a"])
        pause()
        sg.swiglu_fused_grouped_int8(m["A"], m["a"], *W1, *W2, route["offsets"], route["rows"], m["Y"], workspace=m["ws"])
        pause()
        sg.swiglu_quant_int8(m["Y"], m["B"], m["b"])
        pause()
        sg.swiglu_linear_grouped_int8(m["B"], m["b"], *W3, route["offsets"], None, m["Z"], workspace=m["ws"])
        pause()
        sg.swiglu_residual_norm(m["Z"], R, slots=route["slots"], weights=route["weights"], Rout=out[0], H=out[1])
        pause()

    outs = lambda: [(e(T, K), e(T, K, d=BF)) for _ in range(turns)]  # noqa: E731
    want, got = outs(), outs()
    for x, out in zip(ins, want):
        turn(x, *buffers(), out, torch.cuda.synchronize)
    route, m = buffers()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)
        for x, out in zip(ins, got):
            turn(x, route, m, out, lambda: None)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            a[0].zero_(), a[1].zero_()
    _status(sg)


def one_code_a_step(M, N, K, mats, seed):
    """Rows of A with a single one in every M-th step of 128 of K, the rows' steps together all of them; weights
    of +-1; the sums, whole numbers up to 256 for up to 256 M steps.  A step lost or doubled changes a row in every column."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    steps = -(-K // 128)
    per = -(-steps // M)
    assert per <= 256
    step = torch.arange(M, device=DEV)[:, None] + M * torch.arange(per, device=DEV)
    at = torch.where(step < steps, (step * 128 + torch.randint(0, 128, step.shape, generator=gen, device=DEV)).clamp(max=K - 1), -1)
    A = torch.zeros(M, K, dtype=I8, device=DEV)
    for m in range(M):
        A[m, at[m][at[m] >= 0]] = 1
    Ws = [torch.randint(0, 2, (N, K), generator=gen, dtype=I8, device=DEV).mul_(2).sub_(1) for _ in range(mats)]
    sums = []
    for W in Ws:
        picked = W[:, at.clamp(min=0).flatten()].view(N, M, per)
        sums.append((picked * (at >= 0)).sum(2, dtype=torch.int32).t().double())
    return A, Ws, sums


@pytest.mark.parametrize("M,N,K", [(200, 4872, (1 << 17) + 48), (200, 4864, (1 << 20) - 1024), (200, 16, (1 << 20) - 1024),
                                   (40, 264, (1 << 20) - 1024), (300, 24, (1 << 19) + 16)])
def test_every_step_of_a_long_k_counts_once(sg, M, N, K):
    """The persistent and the shared tensor-core forms, under the shortest wait limit: a unit's K takes longer than it."""
    A, (W,), (want,) = one_code_a_step(M, N, K, 1, N)
    one = torch.ones(max(M, N), device=DEV)
    _status(sg)
    sg.swiglu_set_wait_timeout_ns(1_000_000)
    try:
        Z = sg.swiglu_linear_int8(A, one[:M].contiguous(), W, one[:N].contiguous())
    finally:
        sg.swiglu_set_wait_timeout_ns(2_000_000_000)
    _status(sg)
    assert torch.equal(Z.double(), want)


def test_every_step_of_a_long_k_counts_once_fused(sg):
    M, N, K = 200, 2440, (1 << 17) + 48
    A, (W1, W2), (g, u) = one_code_a_step(M, N, K, 2, 3)
    one = torch.ones(N, device=DEV)
    Y = sg.swiglu_fused_int8(A, one[:M].contiguous(), W1, one, W2, one)
    _status(sg)
    want = g * torch.sigmoid(g) * u    # g and u are exact; 2^-19: exp and reciprocal
    assert ((Y.double() - want).abs() <= (2.0**-8 + 2.0**-19) * want.abs() + 1e-37).all()


def test_many_long_units_within_a_short_limit(sg):
    """The finder's wait for 32 units (about 2 ms here, one takes 0.06 ms) has a limit of its own."""
    P, K, N = 85000, 16384, 4096        # 443 row tiles x 16 column tiles: 93 units a pair
    gen = torch.Generator(device="cuda").manual_seed(8)
    A = torch.randint(-127, 128, (P, K), generator=gen, dtype=I8, device=DEV)
    W = torch.randint(-127, 128, (1, N, K), generator=gen, dtype=I8, device=DEV)
    a, w = torch.rand(P, generator=gen, device=DEV) * 0.01, torch.rand(1, N, generator=gen, device=DEV) * 0.01
    off = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    _status(sg)
    sg.swiglu_set_wait_timeout_ns(1_000_000)
    try:
        Z = sg.swiglu_linear_grouped_int8(A, a, W, w, off)
    finally:
        sg.swiglu_set_wait_timeout_ns(2_000_000_000)
    _status(sg)
    for i, j in ((0, 3), (42000, 42002), (P - 3, P)):
        ref, tol = product_ref(A[i:j], a[i:j], [(W, w)], [0, j - i], None)
        assert ((Z[i:j].double() - ref).abs() <= tol).all(), (i, j)


@pytest.mark.parametrize("N,K", [(4872, (1 << 17) + 48), (264, (1 << 18) + 16)])
def test_long_sums_of_one_sign_by_number_of_rows(sg, N, K):
    """Sums to 2^32: up to 8 rows integers, exact; more rows K additions of FP32, each off by 2^-23 of the sum at most."""
    c, d = torch.arange(200, device=DEV) % 128 - 128, torch.arange(N, device=DEV) % 127 - 128
    A, W = (v.to(I8)[:, None].expand(-1, K).contiguous() for v in (c, d))
    one = torch.ones(N, device=DEV)
    exact = (K * c[:, None] * d[None]).double()
    few = sg.swiglu_linear_int8(A[:8], one[:8].contiguous(), W, one)
    assert torch.equal(few, exact[:8].float().to(BF))
    many = sg.swiglu_linear_int8(A, one[:200].contiguous(), W, one)
    _status(sg)
    assert ((many.double() - exact).abs() <= (K * 2.0**-23 + 2.0**-8) * exact).all()
