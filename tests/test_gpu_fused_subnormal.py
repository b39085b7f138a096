"""Blocks whose scale has a few significant bits: amax / 448 in the lowest FP32 subnormals.

With amax = k 2^-149 the scale is round(k / 448) 2^-149, and a quotient v / s reaches 671 (k = 671,
s = 2^-149): codes saturate at +-448, where a cast without saturation gives NaN from 464 on.  All
inputs here make values that are whole multiples of 2^-149 in FP32 exactly, so codes and scales have
one right answer."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import f64

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -149


def expected(k):
    """(code bytes, scales in units of 2^-149) of the 1x128 row blocks of int64 k [rows][cols], in those units.
    Integers below 2^24 are exact in FP32, so k / j below is the IEEE quotient of the two subnormals."""
    rows, cols = k.shape
    nb = (cols + 127) // 128
    p = torch.nn.functional.pad(k, (0, nb * 128 - cols)).view(rows, nb, 128)
    j = torch.round(p.abs().amax(2).double() / 448)          # ties to even, as the FP32 division's
    d = j.unsqueeze(2)
    y = (p.float() / torch.where(d > 0, d, torch.ones_like(d)).float()).clamp(-448, 448)
    y = torch.where(d > 0, y, torch.copysign(torch.zeros_like(y), p.float()))
    q = y.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, nb * 128)[:, :cols]
    return q, j


def check(k, q_row, s_row, q_tok, s_tok, what):
    saturated = False
    for kk, q, s in ((k, q_row, s_row), (k.t(), q_tok, s_tok)):
        want, j = expected(kk.contiguous())
        got = q.cpu().contiguous()
        assert torch.equal(f64(s) / UNIT, j), (what, "scales")
        assert not bool(((got & 0x7F) == 0x7F).any()), (what, "NaN codes", int(((got & 0x7F) == 0x7F).sum()))
        # a product of zeros may carry either sign
        assert bool(((got == want) | (((got | want) & 0x7F) == 0)).all()), (what, "codes")
        saturated |= bool((((got & 0x7F) == 0x7E) & (j.repeat_interleave(128, 1)[:, :got.shape[1]] == 1)).any())
    assert saturated, what      # the case is there: an element past 448 times a scale of one unit


def multiples(tokens, cols, most, seed):
    """Whole numbers of a BF16's eight bits, up to `most` in size: whole blocks near one power of two, so that
    every block has its own largest; the last token and the last column alone in their blocks."""
    gen = torch.Generator().manual_seed(seed)
    k = torch.randint(-most, most + 1, (tokens, cols), generator=gen)
    k = (k.double() * torch.rand((tokens, 1), generator=gen).clamp(min=0.05)).round()
    k[-1] = torch.randint(40, most + 1, (cols,), generator=gen)
    k[:, -1] = torch.randint(40, most + 1, (tokens,), generator=gen)
    return k.float().bfloat16().double()


def lay(t, ld_pad, dev, dtype=torch.bfloat16):
    buf = torch.zeros((t.shape[0], (t.shape[1] + 15) // 16 * 16 + ld_pad), dtype=dtype)
    buf[:, :t.shape[1]] = t
    return buf.to(dev)[:, :t.shape[1]]


@pytest.mark.parametrize("tokens,cols", [(1, 1), (1, 300), (129, 257), (257, 129), (256, 384)])
def test_norm(dev, tokens, cols):
    """z = +-1, so that z r is within 1e-6 of +-1 and z r w rounds back to w = k 2^-149 (k < 4096)."""
    gen = torch.Generator().manual_seed(cols)
    k = torch.randint(0, 4096, (cols,), generator=gen)
    k[: min(cols, 440)] = torch.arange(235, 675)[: min(cols, 440)]
    k[0] = 671
    sign = torch.randint(0, 2, (tokens, cols), generator=gen) * 2 - 1
    x, w = lay(sign.double(), 16, dev), (k.double() * UNIT).float().to(dev)
    z, r, _, qr, sr, qt, st = pf.puro_fp8_rmsnorm_quant_dual(x, w, eps=1e-6)
    a = pf.puro_fp8_rmsnorm_quant_act(x, w, eps=1e-6)
    torch.cuda.synchronize()
    assert float((1 - r).abs().max()) < 1e-6
    check(sign * k, qr, sr, qt, st, "norm")
    assert torch.equal(a[3], qr) and torch.equal(a[4], sr)


@pytest.mark.parametrize("tokens,cols", [(1, 1), (1, 300), (129, 257), (257, 129), (256, 384)])
def test_norm_gradient(dev, tokens, cols):
    """z = 0, r = 1 and w = 2^-14: dx = w dy, with dy = k 2^-133 four times k units."""
    k = multiples(tokens, cols, 900, 7)
    k[0, 0] = 160
    dy, z = lay(k * 2.0 ** -133, 0, dev), torch.zeros((tokens, (cols + 15) // 16 * 16), dtype=torch.bfloat16, device=dev)
    w = torch.full((cols,), 2.0 ** -14, device=dev)
    dx, dw, qr, sr, qt, st = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z[:, :cols], torch.ones((tokens,), device=dev), w)
    torch.cuda.synchronize()
    assert not bool(dw.any())
    check((4 * k).long(), qr, sr, qt, st, "dx")


@pytest.mark.parametrize("tokens,cols", [(1, 1), (1, 300), (129, 257), (257, 129), (256, 384)])
def test_activation_gradient(dev, tokens, cols):
    """gate = up = 2^-13: silu(gate) and up silu'(gate) are 2^-14 times 1 + 1.3e-4 at most, and with dh = k 2^-133
    dup and dgate are 4 k units to within half a unit (k <= 900)."""
    k = multiples(tokens, cols, 900, 8)
    k[0, 0] = 160
    dh = lay(k * 2.0 ** -133, 16, dev)
    g = torch.full((tokens, (cols + 15) // 16 * 16), 2.0 ** -13, dtype=torch.bfloat16, device=dev)[:, :cols]
    got = pf.puro_fp8_swiglu_bwd_quant_dual(dh, g, g)
    torch.cuda.synchronize()
    check((4 * k).long(), *got[0], "dgate")
    check((4 * k).long(), *got[1], "dup")
