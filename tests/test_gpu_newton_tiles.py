"""The orthogonalisation on every tile form: each group's results against 64 bits, and bit for bit those of
each matrix alone (which the smaller forms compute)."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from ns_tiles import GROUPS, TILES, tiles
from test_gpu_newton_schulz import gradient, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [1, 3])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_group(dev, name, steps):
    shapes = GROUPS[name]
    assert tiles(shapes) == TILES[name]
    grads = [gradient(r, c, 40 + i, torch.float32, dev, "normal" if i % 2 else "decay", 16)
             for i, (r, c) in enumerate(shapes)]
    # results into rows wider than they need
    bufs = [torch.full((r, (c + 15) // 16 * 16 + 32), 3.0, dtype=torch.bfloat16, device=dev) for r, c in shapes]
    outs = pf.puro_fp8_newton_schulz_grouped(grads, steps=steps, outs=[b[:, :s[1]] for b, s in zip(bufs, shapes)])
    torch.cuda.synchronize()
    for i, (g, o, b) in enumerate(zip(grads, outs, bufs)):
        assert bool((b[:, g.shape[1]:] == 3).all()), i
        assert torch.equal(o, pf.puro_fp8_newton_schulz_grouped([g], steps=steps)[0]), i
        # two of a shape are one test of the arithmetic and two of the addressing
        if shapes.index(shapes[i]) < i - 1:
            continue
        E, R = reference(g.double(), steps=steps)
        err, norm = float((o.double() - E).norm()), float(E.norm())
        assert err <= 1.25 * float((R - E).norm()) + 2.0 ** -8 * norm, (i, err / norm)
