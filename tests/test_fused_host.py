"""The norm and activation-gradient entry points on the host: bad arguments are refused before any
launch, through the C ABI and the binding; the 64-bit references against central differences."""
import ctypes

import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import norm, norm_bwd, swiglu_bwd

OK, NULL, SHAPE, ALIGN, ENUM, WORKSPACE, VALUE = 0, 1, 2, 3, 4, 5, 8
P = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced (validation fails first)
ODD = ctypes.c_void_p((1 << 20) + 4)
NUL = ctypes.c_void_p(0)
BIG = 1 << 24


def _act(suffix="", x=P, ldx=128, res=NUL, ldres=0, w=P, wdt=0, eps=1e-6, tokens=4, cols=128, z=NUL, ldz=0, rstd=P,
         h=NUL, ldh=0, q=P, ldq=128, s=P):
    return getattr(pf.lib(), "puro_fp8_rmsnorm_quant_act" + suffix)(
        x, ldx, res, ldres, w, wdt, eps, tokens, cols, z, ldz, rstd, h, ldh, q, ldq, s, None)


def _dual(suffix="", x=P, ldx=128, res=NUL, ldres=0, w=P, wdt=0, eps=1e-6, tokens=4, cols=128, z=NUL, ldz=0, rstd=P,
          h=NUL, ldh=0, q=P, ldq=128, s=P, t=1, qt=P, ldqt=16, st=P):
    return getattr(pf.lib(), "puro_fp8_rmsnorm_quant_dual" + suffix)(
        x, ldx, res, ldres, w, wdt, eps, tokens, cols, z, ldz, rstd, h, ldh, q, ldq, s, t, qt, ldqt, st, None)


@pytest.mark.parametrize("suffix", ["", "_pow2"])
@pytest.mark.parametrize("fn", [_act, _dual])
def test_norm_refusals(fn, suffix):
    def call(**kw):
        return fn(suffix, **kw)
    assert call(wdt=2) == ENUM
    assert call(tokens=-1) == SHAPE and call(cols=-1) == SHAPE and call(tokens=BIG) == SHAPE
    assert call(ldx=64) == SHAPE and call(ldq=64) == SHAPE and call(ldx=136) == ALIGN and call(ldq=136) == ALIGN
    for name in ("x", "w", "q", "s"):
        assert call(**{name: NUL}) == NULL, name
    for name in ("x", "w", "q"):
        assert call(**{name: ODD}) == ALIGN, name
    assert call(rstd=ctypes.c_void_p((1 << 20) + 2)) == ALIGN
    # a residual needs z, and both are checked
    assert call(res=P, ldres=128) == SHAPE and call(res=P, ldres=128, ldz=128) == NULL
    assert call(res=P, ldres=64, z=P, ldz=128) == SHAPE and call(res=P, ldres=128, z=ODD, ldz=128) == ALIGN
    assert call(h=P, ldh=64) == SHAPE and call(h=ODD, ldh=128) == ALIGN
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE, eps
    assert call(x=NUL, w=NUL, rstd=NUL, q=NUL, s=NUL, tokens=0) == OK


def test_norm_dual_refusals():
    assert _dual(t=2) == ENUM and _dual(rstd=NUL) == NULL
    assert _dual(qt=NUL) == NULL and _dual(st=NUL) == NULL and _dual(ldqt=0) == SHAPE and _dual(ldqt=24) == ALIGN


def _bwd(suffix="", dy=P, lddy=128, z=P, ldz=128, rstd=P, w=P, wdt=0, dres=NUL, lddres=0, tokens=4, cols=128, dx=P,
         lddx=128, dw=P, acc=0, q=P, ldq=128, s=P, t=1, qt=P, ldqt=16, st=P, ws=P, n=1 << 20):
    return getattr(pf.lib(), "puro_fp8_rmsnorm_bwd_quant_dual" + suffix)(
        dy, lddy, z, ldz, rstd, w, wdt, dres, lddres, tokens, cols, dx, lddx, dw, acc, q, ldq, s, t, qt, ldqt, st, ws,
        n, None)


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_norm_bwd_refusals(suffix):
    def call(**kw):
        return _bwd(suffix, **kw)
    assert call(t=2) == ENUM and call(wdt=7) == ENUM and call(acc=2) == ENUM
    assert call(tokens=-1) == SHAPE and call(cols=BIG) == SHAPE
    for name in ("dy", "z", "rstd", "w", "dx", "dw", "q", "s", "qt", "st"):
        assert call(**{name: NUL}) == NULL, name
    for name in ("dy", "z", "w", "dx", "q", "qt"):
        assert call(**{name: ODD}) == ALIGN, name
    for name in ("lddy", "ldz", "lddx", "ldq"):
        assert call(**{name: 64}) == SHAPE and call(**{name: 136}) == ALIGN, name
    assert call(dres=P, lddres=64) == SHAPE and call(dres=ODD, lddres=128) == ALIGN
    need = pf.puro_fp8_rmsnorm_bwd_workspace_size(4, 128)
    assert need > 0 and call(n=need - 1) == WORKSPACE and call(ws=NUL) == WORKSPACE and call(ws=ODD) == WORKSPACE
    assert call(cols=0, lddy=0, ldz=0, lddx=0, ldq=0, dw=NUL, ws=NUL, n=0) == OK
    assert pf.puro_fp8_rmsnorm_bwd_workspace_size(-1, 4) == 0


def _swb(suffix="", dh=P, lddh=128, g=P, ldg=128, u=P, ldu=128, tokens=4, cols=128, t=1, a=None, b=None):
    return getattr(pf.lib(), "puro_fp8_swiglu_bwd_quant_dual" + suffix)(dh, lddh, g, ldg, u, ldu, tokens, cols, t, a,
                                                                        b, None)


def _out(**kw):
    d = dict(q_row=1 << 20, ldq_row=128, s_row=1 << 20, lds_row=1, q_tok=1 << 20, ldq_tok=16, s_tok=1 << 20, lds_tok=1)
    return pf.QuantDualOut(**{**d, **kw})


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_swiglu_bwd_refusals(suffix):
    good = _out()

    def call(a=good, b=good, **kw):
        return _swb(suffix, a=a, b=b, **kw)
    assert call(t=2) == ENUM and call(a=None) == NULL and call(b=None) == NULL
    assert call(tokens=-1) == SHAPE and call(cols=BIG) == SHAPE
    for name in ("dh", "g", "u"):
        assert call(**{name: NUL}) == NULL and call(**{name: ODD}) == ALIGN, name
    for name in ("lddh", "ldg", "ldu"):
        assert call(**{name: 64}) == SHAPE and call(**{name: 136}) == ALIGN, name
    for bad, want in ((dict(q_row=0), NULL), (dict(s_row=0), NULL), (dict(q_tok=0), NULL), (dict(s_tok=0), NULL),
                      (dict(ldq_row=64), SHAPE), (dict(ldq_tok=0), SHAPE), (dict(lds_row=0), SHAPE),
                      (dict(lds_tok=0), SHAPE), (dict(ldq_row=136), ALIGN), (dict(q_tok=(1 << 20) + 8), ALIGN)):
        assert call(a=_out(**bad)) == want and call(b=_out(**bad)) == want, bad
    assert call(t=0, a=_out(ldq_tok=128, lds_tok=127)) == SHAPE
    assert call(tokens=0) == OK


def test_status_string():
    assert pf.puro_status_string(VALUE) == "scalar argument out of range"


def test_binding_refuses():
    x, w = torch.zeros((4, 128), dtype=torch.bfloat16), torch.ones((128,))
    for call in (lambda: pf.puro_fp8_rmsnorm_quant_act(x, w), lambda: pf.puro_fp8_rmsnorm_quant_dual(x, w),
                 lambda: pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, torch.ones((4,)), w),
                 lambda: pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="x: expected"):
        pf.puro_fp8_rmsnorm_quant_act(x.float(), w)


def _differences(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_references_are_gradients():
    """The 64-bit gradients against central differences of the functions (error below h^2 = 1e-10)."""
    gen = torch.Generator().manual_seed(0)

    def rnd(*s):
        return torch.randn(s, generator=gen, dtype=torch.float64)
    z, w, dy, v, u = rnd(6, 50), 1 + 0.2 * rnd(50), rnd(6, 50), rnd(6, 50), rnd(50)
    r = 1 / torch.sqrt(z.square().mean(1) + 1e-6)
    dx, _, dw, _ = norm_bwd(dy, z, r, w, None)
    assert abs(float((dx * v).sum() - _differences(lambda a: (norm(a, w, 1e-6)[0] * dy).sum(), z, v))) < 1e-7
    assert abs(float((dw * u).sum() - _differences(lambda a: (norm(z, a, 1e-6)[0] * dy).sum(), w, u))) < 1e-7
    dg, du, _, _ = swiglu_bwd(dy, z, v)

    def act(g, p):
        return (torch.nn.functional.silu(g) * p * dy).sum()
    e = rnd(6, 50)
    assert abs(float((dg * e).sum() - _differences(lambda a: act(a, v), z, e))) < 1e-7
    assert abs(float((du * e).sum() - _differences(lambda a: act(z, a), v, e))) < 1e-7
