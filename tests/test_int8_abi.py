"""Refusals of the norm and 8-bit entry points (no GPU: every check returns
before any HIP call) and their bindings."""
import ctypes
import os
import re

import pytest
import torch

import mxfp4_quantized_gemm_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)  # aligned, never read
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)
OK, ENULL, ESHAPE, EMODE, EWS, EALIGN = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def test_types_match_the_header():
    with open(os.path.join(ROOT, "include", "mxfp4.h")) as f:
        text = f.read()
    for name in ("DT_F32", "DT_BF16", "DT_F16"):
        assert int(re.search(rf"\bMXFP4_{name}\s*=\s*(\d+)", text).group(1)) == getattr(mx, name)


def norm(lib, name="mxfp4_rmsnorm", **kw):
    a = dict(x=P, x_ld=64, res=P, res_ld=64, w=P, wt=1, rows=4, cols=64, eps=1e-5, dt=1, h=P, h_ld=64,
             out=P, out_ld=64, stat=P)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values(), NULL)


@pytest.mark.parametrize("name", ["mxfp4_rmsnorm", "mxfp4_rmsnorm_int8"])
def test_norm_refusals(lib, name):
    call = lambda **kw: norm(lib, name, **kw)
    assert call(dt=3) == EMODE
    assert call(dt=-1) == EMODE
    assert call(wt=2) == EMODE                      # neither the rows' type nor fp32
    assert call(dt=0, wt=1) == EMODE
    assert call(rows=-1) == ESHAPE
    assert call(cols=0) == ESHAPE
    assert call(cols=32769, x_ld=40000, res_ld=40000, h_ld=40000, out_ld=40000) == ESHAPE
    assert call(rows=1 << 31) == ESHAPE
    for k in ("x_ld", "res_ld", "h_ld", "out_ld"):
        assert call(**{k: 63}) == ESHAPE, k
        assert call(**{k: 1 << 50}) == ESHAPE, k
    assert call(x=NULL) == ENULL
    assert call(out=NULL) == ENULL
    for k in ("x", "res", "w", "h"):
        assert call(**{k: ODD}) == EALIGN, k
    assert call(wt=0, w=TWO) == EALIGN
    assert call(stat=TWO) == EALIGN
    assert call(rows=0, x=NULL, res=NULL, w=NULL, h=NULL, out=NULL, stat=NULL) == OK
    # pitches of matrices that are not there are not looked at
    assert call(rows=0, res=NULL, res_ld=0, h=NULL, h_ld=0) == OK
    if name.endswith("int8"):
        assert call(stat=NULL) == ENULL
    else:
        assert call(out=ODD) == EALIGN


def test_norm_bwd_refusals(lib):
    need = lib.mxfp4_rmsnorm_bwd_workspace_bytes(4, 64)
    assert need >= 64 * 4
    assert lib.mxfp4_rmsnorm_bwd_workspace_bytes(0, 64) == 0
    assert lib.mxfp4_rmsnorm_bwd_workspace_bytes(4, 0) == 0
    assert lib.mxfp4_rmsnorm_bwd_workspace_bytes(-1, 64) == 0

    def call(**kw):
        a = dict(dy=P, dy_ld=64, dh=P, dh_ld=64, h=P, h_ld=64, w=P, wt=1, rstd=P, rows=4, cols=64, dt=1,
                 dx=P, dx_ld=64, dw=P, ws=P, wsb=need)
        assert not set(kw) - set(a)
        a.update(kw)
        return lib.mxfp4_rmsnorm_bwd(*a.values(), NULL)
    assert call(dt=4) == EMODE
    assert call(wt=2) == EMODE
    assert call(rows=-1) == ESHAPE
    assert call(cols=0) == ESHAPE
    assert call(cols=32769, dy_ld=40000, dh_ld=40000, h_ld=40000, dx_ld=40000) == ESHAPE
    for k in ("dy_ld", "dh_ld", "h_ld", "dx_ld"):
        assert call(**{k: 63}) == ESHAPE, k
    for k in ("dy", "h", "rstd", "dx", "ws"):
        assert call(**{k: NULL}) == ENULL, k
    assert call(wsb=need - 1) == EWS
    for k in ("dy", "dh", "h", "dx", "w", "dw"):
        assert call(**{k: ODD}) == EALIGN, k
    assert call(rstd=TWO) == EALIGN
    assert call(ws=TWO) == EALIGN
    assert call(rows=0, dw=NULL, dy=NULL, h=NULL, dx=NULL, rstd=NULL) == OK


def test_quantize_refusals(lib):
    def call(**kw):
        a = dict(x=P, x_ld=64, gate=P, gate_ld=64, rows=4, cols=64, dt=1, q=P, q_ld=64, s=P)
        assert not set(kw) - set(a)
        a.update(kw)
        return lib.mxfp4_int8_quantize(*a.values(), NULL)
    assert call(dt=7) == EMODE
    assert call(rows=-1) == ESHAPE
    assert call(cols=0) == ESHAPE
    assert call(cols=32769, x_ld=40000, gate_ld=40000, q_ld=40000) == ESHAPE
    for k in ("x_ld", "gate_ld", "q_ld"):
        assert call(**{k: 63}) == ESHAPE, k
    for k in ("x", "q", "s"):
        assert call(**{k: NULL}) == ENULL, k
    assert call(x=ODD) == EALIGN
    assert call(gate=ODD) == EALIGN
    assert call(s=TWO) == EALIGN
    assert call(rows=0, x=NULL, gate=NULL, q=NULL, s=NULL) == OK


def test_gemm_refusals(lib):
    def call(**kw):
        a = dict(A=P, lda=64, sa=P, B=P, ldb=64, sb=P, bias=NULL, M=4, N=8, K=64, C=P, ldc=8, dt=1, ws=P,
                 wsb=1 << 40)
        assert not set(kw) - set(a)
        a.update(kw)
        return lib.mxfp4_int8_gemm(*a.values(), NULL)
    assert call(dt=3) == EMODE
    assert call(M=-1) == ESHAPE
    assert call(N=-1) == ESHAPE
    assert call(K=0) == ESHAPE
    assert call(K=131072, lda=131072, ldb=131072) == ESHAPE   # the int32 sum could overflow
    assert call(lda=63) == ESHAPE
    assert call(ldb=63) == ESHAPE
    assert call(ldc=7) == ESHAPE
    assert call(M=1 << 20, N=1 << 20, ldc=1 << 20) == ESHAPE  # more tiles than a grid has
    assert call(N=1 << 26, ldc=1 << 26) == ESHAPE
    assert call(M=1 << 26) == ESHAPE
    for k in ("A", "sa", "B", "sb", "C"):
        assert call(**{k: NULL}) == ENULL, k
    assert call(sa=TWO) == EALIGN
    assert call(sb=TWO) == EALIGN
    assert call(bias=TWO) == EALIGN
    assert call(C=ODD) == EALIGN
    assert call(C=TWO, dt=0) == EALIGN
    empty = dict(A=NULL, sa=NULL, B=NULL, sb=NULL, C=NULL, ws=NULL, wsb=0)
    assert call(M=0, **empty) == OK
    assert call(N=0, **empty) == OK
    assert lib.mxfp4_int8_gemm_workspace_bytes(4, 8, 0) == 0
    assert lib.mxfp4_int8_gemm_workspace_bytes(0, 8, 64) == 0


def test_wrappers_refuse_cpu_tensors_and_wrong_shapes():
    from mxfp4_quantized_gemm_amd import int8, norm
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU memory"):
        norm.rms_norm(x, w)
    with pytest.raises(ValueError, match="GPU memory"):
        norm.rms_norm_int8(x, w)
    with pytest.raises(ValueError, match="residual"):
        norm.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="one dimension"):
        norm.rms_norm(x, x)
    with pytest.raises(ValueError, match="dimension"):
        norm.rms_norm(x[0, 0])
    with pytest.raises(ValueError, match="GPU memory"):
        int8.int8_quantize(x)
    with pytest.raises(ValueError, match="gate"):
        int8.int8_quantize(x, gate=x[:, :32])
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError, match="GPU memory"):
        int8.int8_gemm(q, s, q, s)
    with pytest.raises(ValueError, match="last dimension"):
        int8.Int8Linear(32, 16)(x)
    with pytest.raises(ValueError, match="columns"):
        int8.int8_linear(x, torch.zeros(8, 100, dtype=torch.int8), s)


def test_calls_without_a_gradient_refuse_to_be_recorded():
    from mxfp4_quantized_gemm_amd import int8, norm
    x = torch.zeros(4, 64, dtype=torch.bfloat16, requires_grad=True)
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.ones(4)
    for call in (lambda: int8.int8_quantize(x), lambda: norm.rms_norm_int8(x), lambda: int8.int8_linear(x, q, s),
                 lambda: int8.int8_quantize(x.detach(), gate=x), lambda: norm.rms_norm_int8(x.detach(), residual=x)):
        with pytest.raises(RuntimeError, match="no gradient"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="GPU memory"):
        int8.int8_quantize(x)
