"""Argument checks of the 8-bit calls and the router by scores (no GPU: the
checks are pure host arithmetic on addresses that are never dereferenced)."""
import pytest
import torch

import swiglu_gemm_transformer_gb300 as sg
from swiglu_gemm_transformer_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sg.lib()


A, B, C, D, E, F, G, H, I, J = (0x10000000 * i for i in range(1, 11))
INV, MIS, UNS, OK = sg.ERR_INVALID_ARG, sg.ERR_MISALIGNED, sg.ERR_UNSUPPORTED, sg.OK


def _route(lib, logits=A, fp32=0, score=1, bias=G, groups=8, kept=4, best=2, renorm=0, scale=1.0, ids=B, weights=C, offsets=D,
           rows=E, slots=F, T=16, E_=64, k=8, ws=None, nbytes=0):
    return lib.swiglu_moe_route_scored(logits, fp32, score, bias, groups, kept, best, renorm, scale, ids, weights, offsets, rows,
                                       slots, T, E_, k, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(E_=0), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(fp32=2), INV), (dict(score=2), INV),
    (dict(renorm=2), INV), (dict(scale=float("nan")), INV), (dict(groups=0), INV), (dict(groups=7), INV), (dict(kept=0), INV),
    (dict(kept=9), INV), (dict(best=0), INV), (dict(best=3), INV), (dict(E_=66), INV),
    (dict(groups=64, kept=16), UNS), (dict(E_=60, groups=6, kept=3), UNS), (dict(E_=2048), UNS), (dict(k=33, kept=8), UNS),
    (dict(T=1 << 30), UNS), (dict(logits=None), INV), (dict(ids=None), INV), (dict(offsets=None), INV),
    (dict(logits=A + 1), MIS), (dict(bias=G + 2), MIS), (dict(slots=F + 2), MIS),
    (dict(ids=A), INV), (dict(weights=G + 4), INV), (dict(offsets=G + 252), INV),   # overlaps
    (dict(T=4096), INV), (dict(T=4096, ws=H, nbytes=16), INV), (dict(T=4096, ws=G - 64, nbytes=1 << 20), INV),
])
def test_route_refusals(lib, kw, want):
    assert _route(lib, **kw) == want


def _quant(lib, X=A, fp32=0, Q=B, scale=C, R=16, K=64):
    return lib.swiglu_quant_int8(X, fp32, Q, scale, R, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), INV), (dict(K=-8), INV), (dict(fp32=2), INV), (dict(X=None), INV), (dict(Q=None), INV), (dict(scale=None), INV),
    (dict(R=1 << 31), UNS), (dict(K=1 << 31), UNS), (dict(K=60), MIS), (dict(X=A + 8), MIS), (dict(Q=B + 4), MIS),
    (dict(scale=C + 2), MIS), (dict(Q=A + 16), INV), (dict(scale=A + 64), INV), (dict(scale=B + 1020), INV),
    (dict(X=B - 2048, fp32=1), INV),
    (dict(R=0), OK),
])
def test_quant_refusals(lib, kw, want):
    assert _quant(lib, **kw) == want


def _product(lib, fused, grouped, A_=A, sa=B, W1=C, s1=D, W2=E, s2=F, off=G, rows=H, Y=I, T=512, P=1024, E_=8, N=64, K=64, ws=J,
             nbytes=1 << 20):
    if grouped:
        if fused:
            return lib.swiglu_fused_grouped_int8(A_, sa, W1, s1, W2, s2, off, rows, Y, T, P, E_, N, K, ws, nbytes, None)
        return lib.swiglu_linear_grouped_int8(A_, sa, W1, s1, off, rows, Y, T, P, E_, N, K, ws, nbytes, None)
    if fused:
        return lib.swiglu_fused_int8(A_, sa, W1, s1, W2, s2, Y, T, N, K, ws, nbytes, None)
    return lib.swiglu_linear_int8(A_, sa, W1, s1, Y, T, N, K, ws, nbytes, None)


def test_workspace_size(lib):
    size = lib.swiglu_int8_workspace_size
    assert size(512, 1024, 8, 64, 64, 0) == 512 * 64 * 2   # A's rows
    assert size(1024, 512, 8, 64, 64, 1) == 512 * 64 * 2   # the places'
    assert size(512, 512, 0, 64, 64, 1) == 512 * 64 * 2    # dense
    for args in ((1, 8, 64, 64, 64, 0), (8, 8, 0, 64, 64, 1), (0, 512, 8, 64, 64, 0), (512, 0, 8, 64, 64, 0), (512, 512, 8, 64, 0, 0),
                 (512, 512, 8, 0, 64, 0), (-1, 512, 8, 64, 64, 0), (512, -1, 8, 64, 64, 0), (512, 512, 8, 64, -16, 0), (512, 512, -1, 64, 64, 0),
                 (1 << 31, 512, 8, 64, 64, 0), (512, 1 << 31, 8, 64, 64, 0), (512, 512, 8, 64, 1 << 20, 0), (512, 512, 1025, 64, 64, 0),
                 (512, 512, 8, 1 << 31, 64, 0)):
        assert size(*args) == 0


FUSED = pytest.mark.parametrize("fused", [True, False], ids=["fused", "linear"])
GROUPED = pytest.mark.parametrize("grouped", [True, False], ids=["grouped", "dense"])


@FUSED
@GROUPED
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(N=-8), INV), (dict(K=-16), INV), (dict(A_=None), INV), (dict(sa=None), INV), (dict(W1=None), INV),
    (dict(s1=None), INV), (dict(Y=None), INV), (dict(T=1 << 31), UNS), (dict(N=1 << 31), UNS), (dict(K=1 << 22), UNS),
    (dict(N=1 << 20, K=1 << 21), UNS), (dict(N=60), MIS), (dict(K=56), MIS), (dict(A_=A + 8), MIS), (dict(W1=C + 8), MIS),
    (dict(sa=B + 2), MIS), (dict(s1=D + 1), MIS), (dict(Y=I + 8), MIS),
    (dict(Y=A), INV), (dict(Y=B - 64), INV), (dict(Y=C + 64), INV), (dict(Y=D), INV),   # overlaps
    (dict(ws=None), INV), (dict(nbytes=512 * 64 * 2 - 1), INV), (dict(ws=J + 8), MIS), (dict(ws=A), INV), (dict(ws=I - 64), INV),
    (dict(ws=B - 4096), INV), (dict(ws=C + 64), INV), (dict(ws=D), INV),
    (dict(N=0), OK),
])
def test_product_refusals(lib, fused, grouped, kw, want):
    assert _product(lib, fused, grouped, **kw) == want


@FUSED
@pytest.mark.parametrize("kw,want", [
    (dict(P=-1), INV), (dict(E_=0), INV), (dict(off=None), INV), (dict(rows=None), INV), (dict(E_=1025), UNS), (dict(P=1 << 31), UNS),
    (dict(P=(1 << 31) - 256), UNS), (dict(N=(1 << 31) - 256, K=16), UNS), (dict(off=G + 2), MIS), (dict(rows=H + 1), MIS),
    (dict(Y=G - 64), INV), (dict(Y=H), INV), (dict(P=0), OK),
])
def test_grouped_refusals(lib, fused, kw, want):
    assert _product(lib, fused, True, **kw) == want


@GROUPED
@pytest.mark.parametrize("kw,want", [(dict(W2=None), INV), (dict(s2=None), INV), (dict(W2=E + 8), MIS), (dict(s2=F + 2), MIS),
                                     (dict(Y=E), INV), (dict(Y=F - 16), INV)])
def test_fused_needs_both_weights(lib, grouped, kw, want):
    assert _product(lib, True, grouped, **kw) == want


def test_dense_without_rows(lib):
    assert _product(lib, True, False, T=0) == OK


def test_python_binding_refuses_cpu_tensors_and_types(lib):
    x, q = torch.zeros(8, 16), torch.zeros(8, 16, dtype=torch.int8)
    s, off = torch.zeros(8), torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros(2, 8, 16, dtype=torch.int8), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        sg.swiglu_moe_route_scored(x, 2)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        sg.swiglu_quant_int8(x.half())
    for call in (lambda: sg.swiglu_quant_int8(x), lambda: sg.swiglu_linear_int8(q, s, q, s), lambda: sg.swiglu_fused_int8(q, s, q, s, q, s),
                 lambda: sg.swiglu_linear_grouped_int8(q, s, w, ws, off), lambda: sg.swiglu_fused_grouped_int8(q, s, w, ws, w, ws, off)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        sg.swiglu_linear_grouped_int8(q, s, w, ws, None)
    with pytest.raises(TypeError):
        sg.swiglu_fused_int8(q, s, q, s, None, s)
    with pytest.raises(TypeError):
        sg.swiglu_fused_grouped_int8(q, s, w, ws, w, ws, None)


@pytest.mark.parametrize("fused", [0, 1])
@pytest.mark.parametrize("args", [(512, 512, 8, 60, 64), (512, 512, 8, 64, 56), (512, 512, 0, 64, 8), (512, 300, 0, 64, 64),
                                  (512, 512, 8, 1 << 22, 1 << 18), (512, 512, 0, (1 << 31) - 512, 1 << 10), (512, 512, 1, 1 << 24, 1 << 16)])
def test_workspace_size_is_zero_for_refused_sizes(lib, args, fused):
    """Columns and K of other multiples, matrices of 2^40 bytes, a dense call of two sizes of rows."""
    assert lib.swiglu_int8_workspace_size(*args, fused) == 0


def test_workspace_size_of_the_largest_matrices(lib):
    size = lib.swiglu_int8_workspace_size
    assert size(512, 512, 8, (1 << 20) + 1024, (1 << 20) - 1024, 0) == 512 * ((1 << 20) - 1024) * 2   # N K = 2^40 - 2^20
    assert size(512, 512, 8, (1 << 20) + 1032, (1 << 20) - 1024, 0) == 0


@pytest.mark.parametrize("E,N,K,fused,few,many", [   # (places at which either form was measured at least 10 % faster)
    (1, 1024, 2048, 1, (2, 16), (32, 64, 128)), (1, 4864, 896, 1, (2, 4), (12, 32, 128)), (1, 8192, 8192, 0, (2, 4), (12, 32, 128)),
    (1, 18944, 3584, 1, (1,), (4, 8, 16, 32, 128)), (2, 18944, 3584, 1, (1,), (8, 16, 32)), (8, 4864, 896, 1, (2, 4), (12, 16, 32)),
    (8, 896, 4864, 0, (8, 32), (64, 128)), (8, 3584, 18944, 0, (2, 24, 32), (96, 128)), (8, 14336, 4096, 1, (2,), (16, 32)),
    (64, 1024, 2048, 1, (8, 32), (96, 128)), (64, 4864, 896, 1, (8,), (24, 32, 64)), (256, 2048, 1024, 0, (8, 64), (96, 128))])
def test_grouped_calls_of_few_places_take_the_faster_form(lib, E, N, K, fused, few, many):
    """The form of few rows needs no workspace."""
    for P in few:
        assert lib.swiglu_int8_workspace_size(P, P, E, N, K, fused) == 0, P
    for P in many:
        assert lib.swiglu_int8_workspace_size(P, P, E, N, K, fused) == P * K * 2, P
