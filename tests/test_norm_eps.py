"""eps of the norm on the host: normal FP32 numbers only."""
import ctypes

import pytest

import blockwise_fp8_gemm_amd as pf

OK, VALUE = 0, 8


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_eps(suffix):
    nul = ctypes.c_void_p(0)

    def call(eps):      # no tokens: nothing is launched
        return getattr(pf.lib(), "puro_fp8_rmsnorm_quant_act" + suffix)(
            nul, 128, nul, 0, nul, 0, eps, 0, 128, nul, 0, nul, nul, 0, nul, 128, nul, None)
    for eps in (2.0 ** -126, 1e-12, 1e-6, 1.0, 1e30):
        assert call(eps) == OK, eps
    for eps in (2.0 ** -126 * (1 - 2.0 ** -23), 1e-40, 2.0 ** -149, 0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps) == VALUE, eps
