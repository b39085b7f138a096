"""GPU parity of the Newton-Schulz orthogonalisation against the 64-bit iteration.

The tolerance comes from the number formats alone: the same iteration in 64 bits with every value
rounded where the kernels round it (FP16 operands, X as a sum of two FP16 numbers, B's diagonal
kept apart) is so far from the unrounded one; the result may be 1.25 times as far (Frobenius), as
FP32 sums move single FP16 roundings, plus the BF16 rounding of the result (half a step, 2^-8
relative).  Single elements are checked after one step, against a bound that adds every rounding's
largest effect (test_one_step_by_element)."""
import math

import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import f64

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)


def _half(t):
    return t.float().half().double()


def reference(G, steps=5, coef=COEF, eps=1e-7):
    """(exact, emulated) results for a float64 G."""
    tall = G.shape[0] > G.shape[1]
    X = (G.t() if tall else G).contiguous()
    X = X / (torch.linalg.vector_norm(X) + eps)
    s, sa = 2.0 ** round(0.5 * math.log2(X.shape[1])), 1024.0
    a, b, c = coef
    E, R = X.clone(), (X * s).float().double()
    for _ in range(steps):
        A = E @ E.t()
        E = a * E + (b * A + c * A @ A) @ E
        hi = _half(R)
        both = hi + _half(R - hi)
        A = _half(hi @ hi.t() * (sa / s ** 2))
        B = b * A + c / sa * (A @ A)
        d = torch.diagonal(B).clone()
        B = _half(B - torch.diag(d))
        R = (a + d / sa)[:, None] * both + B @ hi / sa
    R = R / s
    return (E.t(), R.t()) if tall else (E, R)


def check(out, G, **kw):
    E, R = reference(f64(G), **kw)
    got = f64(out)
    assert got.shape == E.shape and bool(torch.isfinite(got).all())
    norm = float(E.norm())
    err = float((got - E).norm())
    assert err <= 1.25 * float((R - E).norm()) + 2.0 ** -8 * norm, (err / norm, float((R - E).norm()) / norm)


def gradient(rows, cols, seed, dtype, device, kind="decay", pad=0):
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn((rows, cols), generator=gen)
    if kind == "decay":      # strong directions over a floor
        k = min(8, rows, cols)
        g = 0.05 * g + torch.randn((rows, k), generator=gen) @ torch.randn((k, cols), generator=gen)
    buf = torch.full((rows, (cols + 15) // 16 * 16 + pad), float("nan"), dtype=dtype)
    buf[:, :cols] = (g * 1e-4).to(dtype)
    return buf.to(device)[:, :cols]


SIZES = [(1, 1), (1, 300), (300, 1), (16, 16), (64, 64), (127, 129), (129, 64), (128, 640), (260, 1000), (513, 300),
         (512, 512), (768, 1280)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "decay"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_single(dev, rows, cols, kind, dtype):
    g = gradient(rows, cols, rows * 7 + cols, dtype, dev, kind, 16)
    out, = pf.puro_fp8_newton_schulz_grouped([g])
    torch.cuda.synchronize()
    check(out, g)


@pytest.mark.parametrize("rows,cols", SIZES)
def test_one_step_by_element(dev, rows, cols):
    """Every element after one step.  With u = 2^-11 (half a step of FP16) and f = K 2^-24 for an FP32 sum of
    K terms, to first order:
      hi:  u |X|                    hi + lo: 2^-21 |X| (22 bits, and the FP32 scaling)
      A:   (2 u + f) |X||X|^T + u |A|
      B:   |b| dA + |c| (2 |A| dA + f |A||A|), off the diagonal + u |B|
      X':  |a + d| 2^-21 |X| + dd |X| + (dB + u |B|) |X| + f |B||X|
    FP16's subnormals (spacing 2^-24) add less than 2^-18 of the scaled entries' products; the factor 1.02
    covers the second order.  BF16 rounds once."""
    g = gradient(rows, cols, rows + cols, torch.float32, dev, "normal", 16)
    out, = pf.puro_fp8_newton_schulz_grouped([g], steps=1)
    torch.cuda.synchronize()
    G = f64(g)
    X = (G.t() if rows > cols else G).contiguous()
    X = X / (torch.linalg.vector_norm(X) + 1e-7)
    a, b, c = COEF
    u, fn, fm = 2.0 ** -11, X.shape[1] * 2.0 ** -24, X.shape[0] * 2.0 ** -24
    A = X @ X.t()
    B = b * A + c * A @ A
    E = a * X + B @ X
    P, Q = X.abs(), A.abs()
    dA = (2 * u + fn) * P @ P.t() + u * Q
    dB = abs(b) * dA + abs(c) * (2 * Q @ dA + fm * Q @ Q)
    d = torch.diagonal(B)
    O = (B - torch.diag(d)).abs()
    dX = (a + d).abs()[:, None] * 2.0 ** -21 * P + dB @ P + 2 * u * O @ P + fm * O @ P
    tol = 1.02 * dX + 2.0 ** -18 / X.shape[1] ** 0.5 + 2.0 ** -8 * (E.abs() + 1.02 * dX)
    if rows > cols:
        E, tol = E.t(), tol.t()
    off = (f64(out) - E).abs() - tol
    assert bool((off <= 0).all()), (float(off.max()), float(E.abs().max()))


def test_grouped_equals_single_and_repeats(dev):
    """Wide, tall, square and empty matrices in one call (more than one launch holds), as alone, bit for bit."""
    shapes = [(512, 256), (256, 512), (64, 64), (0, 128), (130, 700), (300, 1)] * 3 + [(512, 1024)]
    grads = [gradient(r, c, 100 + i, torch.float32, dev) for i, (r, c) in enumerate(shapes)]
    outs = pf.puro_fp8_newton_schulz_grouped(grads)
    again = pf.puro_fp8_newton_schulz_grouped(grads)
    torch.cuda.synchronize()
    for g, a, b in zip(grads, outs, again):
        assert torch.equal(a, b)
        assert torch.equal(a, pf.puro_fp8_newton_schulz_grouped([g])[0])


@pytest.mark.parametrize("count", [1, 2, 4, 8])
def test_every_tile_size_gives_the_same_bits(dev, count):
    """More equal matrices in a call move its products to larger tiles: the same results, bit for bit."""
    shape = (2048, 512)
    g = gradient(*shape, 901, torch.float32, dev)
    one, = pf.puro_fp8_newton_schulz_grouped([g], steps=2)
    outs = pf.puro_fp8_newton_schulz_grouped([g] * count + [gradient(1024, 1024, 902, torch.float32, dev)], steps=2)
    torch.cuda.synchronize()
    check(one, g, steps=2)
    for o in outs[:count]:
        assert torch.equal(o, one)


def test_whole_tiles_of_256(dev):
    """Sizes that the 256 x 256 tiles take, in a group and alone."""
    grads = [gradient(r, c, 200 + i, torch.float32, dev) for i, (r, c) in enumerate([(1024, 512), (512, 512),
                                                                                    (256, 1792)])]
    for g, o in zip(grads, pf.puro_fp8_newton_schulz_grouped(grads)):
        check(o, g)


def test_transposed_input_gives_the_transpose(dev):
    g = gradient(300, 200, 301, torch.float32, dev)
    t = torch.zeros((200, 304), device=dev)[:, :300]
    t.copy_(g.t())
    a, b = pf.puro_fp8_newton_schulz_grouped([g, t])
    torch.cuda.synchronize()
    assert torch.equal(a, b.t())


def test_degenerate_matrices(dev):
    """Zeros give zeros; a rank-one matrix and zero rows keep their null space at zero."""
    z = torch.zeros((130, 256), device=dev)
    r1 = torch.randn((200, 1), device=dev) @ torch.randn((1, 144), device=dev)
    zr = gradient(128, 256, 401, torch.float32, dev, "normal")
    zr[5:40] = 0
    a, b, c = pf.puro_fp8_newton_schulz_grouped([z, r1, zr])
    torch.cuda.synchronize()
    assert not bool(a.any()) and not bool(c[5:40].any())
    check(b, r1)
    check(c, zr)


@pytest.mark.parametrize("scale", [1e-25, 1e20])
def test_magnitudes(dev, scale):
    g = gradient(96, 224, 501, torch.float32, dev) * scale
    out, = pf.puro_fp8_newton_schulz_grouped([g], eps=1e-37)
    torch.cuda.synchronize()
    check(out, g, eps=1e-37)


def test_coefficients_and_steps(dev):
    """A cubic of one's own, one step, and a triple per step."""
    g = gradient(96, 224, 601, torch.float32, dev)
    cubic = (1.5, -0.5, 0.0)
    for steps in (1, 2, 8):
        out, = pf.puro_fp8_newton_schulz_grouped([g], steps=steps, coefficients=cubic)
        check(out, g, steps=steps, coef=cubic)
    a, = pf.puro_fp8_newton_schulz_grouped([g], steps=3, coefficients=[COEF] * 3)
    b, = pf.puro_fp8_newton_schulz_grouped([g], steps=3, coefficients=COEF)
    assert torch.equal(a, b)


def test_singular_values_are_driven_to_one(dev):
    out, = pf.puro_fp8_newton_schulz_grouped([gradient(256, 1024, 701, torch.float32, dev, "normal")])
    s = torch.linalg.svdvals(f64(out))
    # the quintic's fixed interval, wider by the result's BF16 rounding (its norm times 2^-8)
    assert 0.65 <= float(s.min()) and float(s.max()) <= 1.25, (float(s.min()), float(s.max()))


def test_given_outputs_and_workspace(dev):
    g = gradient(130, 200, 801, torch.float32, dev)
    buf = torch.full((130, 240), 3.0, dtype=torch.bfloat16, device=dev)
    need = pf.puro_fp8_newton_schulz_workspace_size([(130, 200)])
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=dev)   # what it held does not matter
    out, = pf.puro_fp8_newton_schulz_grouped([g], outs=[buf[:, :200]], workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((buf[:, 200:] == 3).all()) and bool((ws[need:] == 0xA5).all())
    assert torch.equal(out, pf.puro_fp8_newton_schulz_grouped([g])[0])
