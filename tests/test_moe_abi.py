"""Argument checks of the sparse MLP block's entry points (no GPU: the checks
are pure host arithmetic on addresses that are never dereferenced)."""
import pytest
import torch

import swiglu_gemm_transformer_gb300 as sg
from swiglu_gemm_transformer_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sg.lib()


A, B, C, D, E, F, G, H = (0x10000000 * i for i in range(1, 9))
INV, MIS, UNS, OK = sg.ERR_INVALID_ARG, sg.ERR_MISALIGNED, sg.ERR_UNSUPPORTED, sg.OK


def test_route_workspace_size(lib):
    assert lib.swiglu_moe_route_workspace_size(1, 64, 8) == 0
    n = lib.swiglu_moe_route_workspace_size(16384, 64, 8)
    assert n > 0 and n % (64 * 4) == 0
    assert lib.swiglu_moe_route_workspace_size(0, 64, 8) == 0
    assert lib.swiglu_moe_route_workspace_size(-5, 64, 8) == 0


@pytest.mark.parametrize("T,E_,k", [((1 << 63) - 1, 1, 1), ((1 << 63) - 1, 1 << 62, 1), (1 << 40, 1024, 32), (1 << 26, 64, 33),
                                    (4096, 1025, 8), (4096, 1 << 62, 8), (1 << 31, 8, 1)])
def test_route_workspace_size_of_calls_that_are_refused(lib, T, E_, k):
    assert lib.swiglu_moe_route_workspace_size(T, E_, k) == 0
    assert _route(lib, T=T, E_=E_, k=k) == (INV if k > E_ else UNS)


def test_route_workspace_size_of_the_most_tokens(lib):
    T = (1 << 31) - 1
    assert lib.swiglu_moe_route_workspace_size(T, 1024, 1) == -(-T // 128) * 1024 * 4


def _route(lib, logits=A, fp32=0, renorm=0, scale=1.0, ids=B, weights=C, offsets=D, rows=E, slots=F,
           T=16, E_=64, k=8, ws=None, nbytes=0):
    return lib.swiglu_moe_route(logits, fp32, renorm, scale, ids, weights, offsets, rows, slots, T, E_, k,
                                ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(E_=0), INV), (dict(k=0), INV), (dict(k=65), INV), (dict(fp32=2), INV),
    (dict(renorm=2), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(weights=None), INV), (dict(offsets=None), INV),
    (dict(rows=None), INV), (dict(slots=None), INV),
    (dict(E_=1025), UNS), (dict(E_=64, k=33), UNS), (dict(T=1 << 30), UNS),
    (dict(logits=A + 1), MIS), (dict(logits=A + 2, fp32=1), MIS), (dict(ids=B + 2), MIS),
    (dict(offsets=D + 1), MIS),
    (dict(ids=A), INV), (dict(rows=F + 4), INV), (dict(weights=D), INV),     # overlaps
    (dict(T=4096), INV),                                                     # no workspace
    (dict(T=4096, ws=G, nbytes=16), INV),
    (dict(T=4096, ws=A, nbytes=1 << 20), INV),                               # workspace over the logits
])
def test_route_refusals(lib, kw, want):
    assert _route(lib, **kw) == want


def _grouped(lib, fused, A_=A, W1=B, W2=C, off=D, rows=E, Y=F, T=64, P=128, E_=8, N=64, K=64):
    if fused:
        return lib.swiglu_fused_grouped(A_, W1, W2, off, rows, Y, T, P, E_, N, K, None)
    return lib.swiglu_linear_grouped(A_, W1, off, rows, Y, T, P, E_, N, K, None)


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(P=-1), INV), (dict(E_=0), INV), (dict(N=-8), INV), (dict(K=-8), INV),
    (dict(A_=None), INV), (dict(W1=None), INV), (dict(off=None), INV), (dict(Y=None), INV),
    (dict(rows=None), INV),                       # T != P
    (dict(E_=1025), UNS), (dict(P=1 << 31), UNS), (dict(N=1 << 31), UNS),
    (dict(N=1 << 24, K=1 << 24), UNS),
    (dict(N=60), MIS), (dict(K=60), MIS), (dict(A_=A + 8), MIS), (dict(W1=B + 2), MIS),
    (dict(off=D + 2), MIS), (dict(rows=E + 1), MIS), (dict(Y=F + 8), MIS),
    (dict(Y=A), INV), (dict(Y=B + 64), INV), (dict(Y=D - 64), INV), (dict(Y=E), INV),   # overlaps
    (dict(P=0), OK), (dict(N=0), OK),
])
def test_grouped_refusals(lib, fused, kw, want):
    assert _grouped(lib, fused, **kw) == want


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("kw", [dict(P=(1 << 31) - 1), dict(P=(1 << 31) - 256), dict(N=(1 << 31) - 8, K=8),
                                dict(N=(1 << 31) - 256, K=8)])
def test_grouped_refuses_sizes_whose_last_tile_passes_32_bits(lib, fused, kw):
    assert _grouped(lib, fused, **kw) == UNS


def test_grouped_needs_both_weights(lib):
    assert _grouped(lib, True, W2=None) == INV
    assert _grouped(lib, True, W2=C + 4) == MIS
    assert _grouped(lib, True, Y=C) == INV


def _norm(lib, Z=A, slots=None, weights=None, R=B, r32=0, post=1, gpost=C, gate=None, gs=0, scale=1.0,
          gpre=D, eps=1e-6, Rout=E, Hh=F, T=16, P=16, k=0, Dd=64):
    return lib.swiglu_residual_norm(Z, slots, weights, R, r32, post, gpost, gate, gs, scale, gpre, eps, Rout,
                                    Hh, T, P, k, Dd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(P=-1), INV), (dict(k=-1), INV), (dict(Dd=-8), INV), (dict(gs=-8), INV),
    (dict(r32=2), INV), (dict(post=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(Z=None), INV), (dict(R=None), INV), (dict(Rout=None), INV),
    (dict(P=32), INV),                                   # no slots, P != T
    (dict(slots=G, k=2, P=32), INV),                     # slots without weights
    (dict(post=0), INV),                                 # gamma_post without the norm
    (dict(gate=G, gs=32), INV),                          # rows of the gate overlap
    (dict(Dd=32776), UNS), (dict(T=1 << 31, P=1 << 31), UNS),
    (dict(Dd=60), MIS), (dict(gate=G, gs=68), MIS), (dict(Z=A + 8), MIS), (dict(R=B + 4), MIS),
    (dict(gpost=C + 2), MIS), (dict(Hh=F + 2), MIS), (dict(slots=G + 1, weights=H, k=2, P=32), MIS),
    (dict(Rout=A), INV), (dict(Rout=B + 16), INV), (dict(Hh=B), INV), (dict(Hh=E + 16), INV),
    (dict(Hh=A + 32), INV), (dict(gate=F, gs=64), INV),
    (dict(T=0, P=0), OK), (dict(Dd=0), OK),
])
def test_residual_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def test_python_binding_refuses_cpu_tensors_and_types(lib):
    x = torch.zeros(8, 8, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sg.swiglu_moe_route(x, 2)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        sg.swiglu_moe_route(x.half(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        sg.swiglu_fused_grouped(x, w, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        sg.swiglu_linear_grouped(x, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        sg.swiglu_residual_norm(x, x)
