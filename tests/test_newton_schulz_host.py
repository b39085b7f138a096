"""The Newton-Schulz entry point on the host: bad arguments are refused before any launch."""
import ctypes

import pytest
import torch

import blockwise_fp8_gemm_amd as pf

OK, NULL, SHAPE, ALIGN, ENUM, WORKSPACE, VALUE = 0, 1, 2, 3, 4, 5, 8
A = 1 << 20


def _call(dt=0, items=None, count=None, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7, ws=A, n=1 << 30, **kw):
    d = dict(g=A, rows=64, cols=64, ldg=64, o=A, ldo=64)
    if items is None:
        items = [pf.NewtonSchulzDesc(*[{**d, **kw}[k] for k in ("g", "rows", "cols", "ldg", "o", "ldo")])]
    arr = (pf.NewtonSchulzDesc * max(len(items), 1))(*items)
    c = (ctypes.c_float * (3 * max(steps, 1)))(*(list(coef) * max(steps, 1))) if coef is not None else None
    return pf.lib().puro_fp8_newton_schulz_grouped(dt, arr, len(items) if count is None else count, steps, c, eps,
                                                   ctypes.c_void_p(ws), n, None)


def test_refusals():
    assert _call(dt=2) == ENUM
    assert _call(count=-1) == SHAPE and _call(count=4097) == SHAPE
    assert _call(coef=None) == NULL and _call(g=0) == NULL and _call(o=0) == NULL
    for name in ("rows", "cols"):
        assert _call(**{name: -1}) == SHAPE and _call(**{name: 16385, "ldg": 1 << 20, "ldo": 1 << 20}) == SHAPE
    for name in ("ldg", "ldo"):
        assert _call(**{name: 48}) == SHAPE and _call(**{name: 72}) == ALIGN
    assert _call(g=A + 4) == ALIGN and _call(o=A + 8) == ALIGN
    need = pf.puro_fp8_newton_schulz_workspace_size([(64, 64)])
    assert need > 0 and _call(n=need - 1) == WORKSPACE and _call(ws=0) == WORKSPACE and _call(ws=A + 16) == WORKSPACE
    assert _call(items=[]) == OK and _call(rows=0, g=0, o=0, ws=0, n=0) == OK


def test_values_out_of_range():
    for steps in (0, -1, 33):
        assert _call(steps=steps) == VALUE
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _call(eps=eps) == VALUE
    for coef in ((float("nan"), 0, 0), (float("inf"), 0, 0), (2.1, 0, 0), (1, 40, 0), (1, 0, 40), (0, 0, 2.5),
                 (8.0, -9.0, 2.0), (0, 6.0, 0)):
        assert _call(coef=coef) == VALUE, coef
    # (8, -9, 2) ends at 1 for s = 1 and passes 2 on the way there; these stay inside on the whole interval
    for coef in ((1.5, -0.5, 0.0), (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375), (1, 0, 0)):
        assert _call(coef=coef, rows=0) == OK, coef


def test_workspace_size():
    size = pf.puro_fp8_newton_schulz_workspace_size
    assert size([]) == 0 and size([(-1, 4)]) == 0 and size([(16385, 4)]) == 0 and size([(0, 5)]) == 0
    assert size([(64, 200)]) == size([(200, 64)])
    assert size([(64, 64)] * 17) == size([(64, 64)] * 16) == 16 * size([(64, 64)])


def test_binding_refuses():
    g = torch.zeros((16, 16))
    with pytest.raises(ValueError, match="on the GPU"):
        pf.puro_fp8_newton_schulz_grouped([g])
    with pytest.raises(ValueError, match="one per step"):
        pf.puro_fp8_newton_schulz_grouped([g], steps=2, coefficients=[(1, 0, 0)])
    with pytest.raises(ValueError, match="one entry per gradient"):
        pf.puro_fp8_newton_schulz_grouped([g], outs=[])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        pf.puro_fp8_newton_schulz_grouped([g.half()])
    assert pf.puro_fp8_newton_schulz_grouped([]) == []
