"""What the header promises of five steps of the usual quintic: within 2e-3 (relative Frobenius) of the exact
chain before the result's rounding to BF16, on spectra that gradients and momenta have."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from test_gpu_newton_schulz import COEF

pytestmark = pytest.mark.gpu


def exact(G, steps=5, eps=1e-7):
    """The chain in 64 bits, on the tensor's device."""
    tall = G.shape[0] > G.shape[1]
    X = (G.t() if tall else G).contiguous()
    X = X / (torch.linalg.vector_norm(X) + eps)
    a, b, c = COEF
    for _ in range(steps):
        A = X @ X.t().contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if tall else X


def spectrum(kind, rows, cols, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=gen, device=dev)
    m = min(rows, cols)
    if kind == "normal":
        return rnd(rows, cols)
    if kind == "decay":                 # a few strong directions over a floor
        return 0.05 * rnd(rows, cols) + rnd(rows, 8) @ rnd(8, cols)
    if kind == "rows":                  # rows of very different size
        return rnd(rows, cols) * torch.exp(2 * rnd(rows, 1))
    if kind == "low rank":              # rank 32 over a floor of 1e-3 of it
        return 1e-3 * rnd(rows, cols) + rnd(rows, 32) @ rnd(32, cols) / 32 ** 0.5
    power = {"power 0.5": -0.5, "power 1": -1.0}[kind]
    u, v = (torch.linalg.qr(rnd(n, m))[0] for n in (rows, cols))
    s = torch.arange(1, m + 1, device=dev, dtype=torch.float32) ** power
    return (u * s) @ v.t().contiguous()


def half_step(o):
    """Half a BF16 step at each element (2^-9 of its power of two)."""
    _, e = torch.frexp(o.double())
    return torch.where(o == 0, torch.zeros_like(o, dtype=torch.float64), torch.ldexp(torch.ones_like(o, dtype=torch.float64), e - 9))


@pytest.mark.parametrize("rows,cols", [(384, 1152), (700, 300), (1024, 2048), (2048, 2048), (6144, 2048)])
@pytest.mark.parametrize("kind", ["normal", "decay", "rows", "low rank", "power 0.5", "power 1"])
def test_five_steps(dev, kind, rows, cols):
    """The rounding to BF16 is at most half a step h of each element and evenly spread over it: its squares add up
    to sum h^2 / 3, with a variance of 4/45 sum h^4; what it has in common with the error before it has a variance
    of 4/3 max h^2 times that error's square.  Six standard deviations are allowed."""
    g = pf.empty_2d(rows, cols, torch.float32, dev).copy_(spectrum(kind, rows, cols, 7, dev))
    out, = pf.puro_fp8_newton_schulz_grouped([g])
    torch.cuda.synchronize()
    E = exact(g.double())
    before = (2e-3 * float(E.norm())) ** 2
    h2 = half_step(out).square()
    spread = (4 / 45 * float(h2.square().sum()) + 4 / 3 * float(h2.max()) * before) ** 0.5
    err = float((out.double() - E).square().sum())
    print("%-10s %5d x %4d: %.2e with the rounding, %.2e before it" % (
        kind, rows, cols, (err / float(E.square().sum())) ** 0.5,
        max(err - float(h2.sum()) / 3, 0) ** 0.5 / float(E.norm())), flush=True)
    assert err <= before + float(h2.sum()) / 3 + 6 * spread, ((err / float(E.square().sum())) ** 0.5)
