"""GPU parity of the norm and its gradient against 64-bit references (tolerances derived there).

Sizes: one token to several token blocks, one column to rows wider than a workgroup holds in
registers, ragged in both extents, padded rows; FP32 and BF16 weights; with and without the
residual; both scale rules and both token-copy layouts; rows that are all zero, rows with one
channel far above the rest, and values whose scales are subnormal."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16, check_blocks, check_dual, close_bf16, f64, norm, norm_bwd

pytestmark = pytest.mark.gpu

EPS = 1e-6
SIZES = [(1, 1), (1, 2048), (2, 128), (3, 130), (127, 129), (128, 128), (130, 512), (257, 384), (300, 1000),
         (129, 8200), (2, 20000)]


def _weight(cols, seed, dtype, device):
    gen = torch.Generator().manual_seed(seed)
    return (1.0 + 0.2 * torch.randn((cols,), generator=gen)).to(dtype).to(device)


def _stream_in(tokens, cols, seed, device, pad):
    """A residual stream: one channel far above the rest, one row all zero."""
    r = bf16(tokens, cols, 2.0, seed, device, pad)
    r[:, cols // 2] *= 100
    return r


def _forward(x, res):
    return f64((x.float() + res.float()).bfloat16()) if res is not None else f64(x)


@pytest.mark.parametrize("pow2", [False, True], ids=["amax", "pow2"])
@pytest.mark.parametrize("residual", [False, True], ids=["x", "x+res"])
@pytest.mark.parametrize("tokens,cols", SIZES)
def test_act(dev, tokens, cols, residual, pow2):
    x = bf16(tokens, cols, 1.0, 11, dev, 16)
    res = _stream_in(tokens, cols, 12, dev, 32) if residual else None
    if tokens > 2:
        x[1] = 0
        if residual:
            res[1] = 0
    w = _weight(cols, 13, torch.bfloat16 if cols % 2 else torch.float32, dev)
    z, rstd, h, q, s = pf.puro_fp8_rmsnorm_quant_act(x, w, res, eps=EPS, store_h=True, pow2=pow2)
    torch.cuda.synchronize()
    zx = _forward(x, res)
    assert torch.equal(f64(z), zx)
    n, tol, r, rel = norm(zx, f64(w), EPS)
    assert bool(((f64(rstd) - r).abs() <= rel * r).all())
    check_blocks(n, tol, q, s, "act", pow2)
    close_bf16(h, n, tol, "h")
    assert pf.puro_fp8_rmsnorm_quant_act(x, w, res, eps=EPS, pow2=pow2)[2] is None


@pytest.mark.parametrize("pow2", [False, True], ids=["amax", "pow2"])
@pytest.mark.parametrize("transpose_out", [True, False], ids=["nt", "tn"])
@pytest.mark.parametrize("tokens,cols", SIZES)
def test_dual(dev, tokens, cols, transpose_out, pow2):
    residual = transpose_out
    x = bf16(tokens, cols, 1.0, 21, dev, 16)
    res = _stream_in(tokens, cols, 22, dev, 0) if residual else None
    if tokens > 2:
        x[1] = 0
        if residual:
            res[1] = 0
    w = _weight(cols, 23, torch.float32 if cols % 2 else torch.bfloat16, dev)
    z, rstd, h, qr, sr, qt, st = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS, transpose_out=transpose_out,
                                                                store_h=True, pow2=pow2)
    torch.cuda.synchronize()
    zx = _forward(x, res)
    assert torch.equal(f64(z), zx)
    n, tol, r, rel = norm(zx, f64(w), EPS)
    assert bool(((f64(rstd) - r).abs() <= rel * r).all())
    check_dual(n, tol, qr, sr, qt, st, "dual", transpose_out, pow2)
    close_bf16(h, n, tol, "h")


@pytest.mark.parametrize("pow2", [False, True], ids=["amax", "pow2"])
@pytest.mark.parametrize("transpose_out", [True, False], ids=["nt", "tn"])
@pytest.mark.parametrize("tokens,cols", SIZES)
def test_backward(dev, tokens, cols, transpose_out, pow2):
    z = _stream_in(tokens, cols, 31, dev, 16)
    dy = bf16(tokens, cols, 1e-3, 32, dev, 0)
    dres = bf16(tokens, cols, 1e-3, 33, dev, 48) if transpose_out else None
    if tokens > 2:
        z[1] = 0
        dy[2] = 0
    w = _weight(cols, 34, torch.float32 if cols % 2 else torch.bfloat16, dev)
    r = torch.rsqrt(z.double().square().mean(1) + EPS).float()
    dx, dw, qr, sr, qt, st = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, dres, transpose_out=transpose_out,
                                                                pow2=pow2)
    torch.cuda.synchronize()
    ex, tol, ew, dtol = norm_bwd(f64(dy), f64(z), f64(r), f64(w), f64(dres) if dres is not None else None)
    close_bf16(dx, ex, tol, "dx")
    assert bool(((f64(dw) - ew).abs() <= dtol).all())
    check_dual(ex, tol, qr, sr, qt, st, "dx", transpose_out, pow2)
    # accumulated into an existing gradient: one more addition
    old = torch.linspace(-1, 1, cols, device=dev)
    acc = old.clone()
    pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, dres, transpose_out=transpose_out, dw=acc, accumulate=True,
                                       pow2=pow2)
    torch.cuda.synchronize()
    assert torch.equal(acc, old + dw)


def test_backward_is_the_forwards_gradient_by_differences(dev):
    """dx and dw against central differences of the forward's 64-bit value along random directions."""
    tokens, cols, h = 5, 200, 1e-5
    z = bf16(tokens, cols, 1.0, 41, dev)
    dy = bf16(tokens, cols, 1.0, 42, dev)
    w = _weight(cols, 43, torch.float32, dev)
    r = torch.rsqrt(z.double().square().mean(1) + EPS).float()
    dx, dw = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w)[:2]
    torch.cuda.synchronize()
    zx, wx, gx = f64(z), f64(w), f64(dy)

    def loss(zz, ww):
        return (norm(zz, ww, EPS)[0] * gx).sum()

    gen = torch.Generator().manual_seed(44)
    for _ in range(4):
        v, u = torch.randn(zx.shape, generator=gen, dtype=torch.float64), torch.randn(wx.shape, generator=gen,
                                                                                      dtype=torch.float64)
        num = (loss(zx + h * v, wx) - loss(zx - h * v, wx)) / (2 * h)
        # BF16 dx: half a step of each term; the differences' own error is below h^2
        assert abs(float((f64(dx) * v).sum() - num)) <= float((f64(dx) * v).abs().sum()) * 2.0 ** -8 + 1e-6
        num = (loss(zx, wx + h * u) - loss(zx, wx - h * u)) / (2 * h)
        assert abs(float((f64(dw) * u).sum() - num)) <= float((f64(dw) * u).abs().sum()) * 64 * 2.0 ** -24 + 1e-6


@pytest.mark.parametrize("mag", [1e-30, 1e-36, 1e-38, 3e-40])
def test_subnormal_scales(dev, mag):
    """Gradients so small that a block's scale is subnormal or zero; dy = 0 leaves dx = dres exactly."""
    tokens, cols = 130, 257
    z = bf16(tokens, cols, 1.0, 51, dev)
    dy = bf16(tokens, cols, 0.0, 53, dev)
    gen = torch.Generator().manual_seed(52)
    dres = (torch.randn((tokens, 272), generator=gen).double() * mag).float().bfloat16().to(dev)[:, :cols]
    r = torch.rsqrt(z.double().square().mean(1) + EPS).float()
    w = torch.ones((cols,), device=dev)
    dx, dw, qr, sr, qt, st = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, z, r, w, dres)
    torch.cuda.synchronize()
    assert torch.equal(dx.float(), dres.float()) and not bool(dw.any())
    check_dual(f64(dres), torch.zeros((tokens, cols), dtype=torch.float64), qr, sr, qt, st, "tiny %g" % mag)


def test_given_outputs_are_written_inside_their_rows_only(dev):
    tokens, cols, ld = 131, 200, 240
    x, res = bf16(tokens, cols, 1.0, 61, dev, 16), bf16(tokens, cols, 1.0, 62, dev, 16)
    w = _weight(cols, 63, torch.float32, dev)
    bufs = {n: torch.full((tokens, ld), 0x5A, dtype=torch.uint8, device=dev) for n in ("q_row",)}
    qt = torch.full((cols, ld), 0x5A, dtype=torch.uint8, device=dev)
    zb, hb = (torch.full((tokens, ld), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ref = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS, store_h=True)
    got = pf.puro_fp8_rmsnorm_quant_dual(x, w, res, eps=EPS, z=zb[:, :cols], h=hb[:, :cols],
                                         q_row=bufs["q_row"][:, :cols], q_tok=qt[:, :tokens])
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert bool((bufs["q_row"][:, cols:] == 0x5A).all()) and bool((qt[:, tokens:] == 0x5A).all())
    assert bool((zb[:, cols:] == 7).all()) and bool((hb[:, cols:] == 7).all())


def test_rows_and_dual_agree_and_repeat(dev):
    """The serving and training forms give the same row codes; equal calls give equal bits."""
    x, res = bf16(300, 640, 1.0, 71, dev), bf16(300, 640, 1.0, 72, dev)
    w = _weight(640, 73, torch.float32, dev)
    a = pf.puro_fp8_rmsnorm_quant_act(x, w, res)
    b = pf.puro_fp8_rmsnorm_quant_dual(x, w, res)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])
    dy = bf16(300, 640, 1.0, 74, dev)
    first = pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, b[0], b[1], w, res)
    for _ in range(5):
        for p, q in zip(first, pf.puro_fp8_rmsnorm_bwd_quant_dual(dy, b[0], b[1], w, res)):
            assert torch.equal(p, q)


def test_no_tokens(dev):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=dev)
    w = torch.ones((256,), device=dev)
    assert pf.puro_fp8_rmsnorm_quant_act(x, w)[3].shape == (0, 256)
    dw = pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, torch.empty((0,), device=dev), w)[1]
    torch.cuda.synchronize()
    assert not bool(dw.any())
    acc = torch.ones((256,), device=dev)
    pf.puro_fp8_rmsnorm_bwd_quant_dual(x, x, torch.empty((0,), device=dev), w, dw=acc, accumulate=True)
    torch.cuda.synchronize()
    assert bool((acc == 1).all())
