"""FP32 tensors whose block scale amax / 448 lies in the lowest FP32 subnormals, byte for byte against the oracle.

A scale of a few units of 2^-149 is rounded by up to half a unit, and a quotient x / s then reaches 671: its
code is +-448, where a cast without saturation gives NaN from 464 on."""
import numpy as np
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
import oracle
from helpers import host, to_dev

pytestmark = pytest.mark.gpu


def tensor(rows, cols, seed):
    """Multiples of 2^-149: every row near a size of its own, amax from 1 to 6,500 units (scales of 0 to 15); the
    last row and column, alone in their blocks at ragged ends, between 225 and 6,500."""
    rng = np.random.default_rng(seed)
    most = np.exp(rng.uniform(np.log(1), np.log(6500), (rows, 1)))
    k = np.rint(rng.uniform(-1, 1, (rows, cols)) * most).astype(np.int64)
    k[-1] = rng.integers(225, 6500, cols)
    k[:, -1] = rng.integers(225, 6500, rows)
    k[0, 0] = 671
    bits = np.abs(k).astype(np.uint32) | ((k < 0).astype(np.uint32) << 31)
    return bits.view(np.float32)


def compare(got, want, what):
    for g, w, part in zip(got, want, ("codes", "scales")):
        g = host(g)
        w = np.asarray(w).reshape(g.shape)
        a, b = (g.view(np.uint32), w.view(np.uint32)) if g.dtype == np.float32 else (g, w)
        assert np.array_equal(a, b), (what, part, int((a != b).sum()))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (129, 257), (257, 129), (256, 384)])
def test_codes_saturate(dev, rows, cols):
    x = tensor(rows, cols, rows + cols)
    d = to_dev(x, dev, (cols + 15) // 16 * 16)
    want = oracle.quant_act(x)
    # the oracle's own codes hold no NaN, and some are saturated at a scale of one unit
    assert not ((want[0] & 0x7F) == 0x7F).any() and ((want[0] & 0x7F) == 0x7E).any()
    compare(pf.puro_fp8_quant_act(d), want, "act")
    compare(pf.puro_fp8_quant_weight(d), oracle.quant_weight(x), "weight")
    compare(pf.puro_fp8_quant_weight_grouped([d])[0], oracle.quant_weight(x), "weight, grouped")
    for t in (True, False):
        tok = oracle.quant_transpose(x, t)
        compare(pf.puro_fp8_quant_transpose(d, t), tok, "transpose")
        both = pf.puro_fp8_quant_dual(d, t)
        compare(both[:2], want, "dual rows")
        compare(both[2:], tok, "dual tokens")
