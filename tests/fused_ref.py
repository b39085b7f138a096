"""64-bit references of the norm, its gradient and the gated activation's gradient, and the
check of codes and scales against values that the kernels form in FP32.

The kernels quantise FP32 values that differ from the exact ones by a few FP32 roundings, so
codes are not compared with one fixed answer: each has to be an E4M3 value nearest to what it
stands for, within the tolerance `tol` (absolute, per element) of the value itself.
"""
import numpy as np
import torch

U = 2.0 ** -24          # half a step of FP32, relative
ROW_THREADS = 256       # the row passes add 8 columns per thread and step


def f64(t):
    return t.detach().double().cpu()


def chain(cols):
    """Additions that one term of a row sum goes through: a thread's own run of columns (8 per
    step), the wave's six exchange steps and the workgroup's waves (at most 16)."""
    return 8 * -(-cols // (8 * ROW_THREADS)) + 6 + 16


def half_step(y):
    """Half the E4M3 spacing at |y| (4 significant bits, spacing 2^-9 below 2^-6)."""
    e = torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6)))
    return torch.exp2(e - 4)


def code_values(q):
    return q.detach().cpu().contiguous().view(torch.float8_e4m3fn).double()


def check_blocks(X, tol, q, s, what, pow2=False):
    """q, s against float64 X [rows][cols] in 1x128 blocks along the rows; tol as X."""
    rows, cols = X.shape
    nb = (cols + 127) // 128
    q, s = code_values(q), f64(s)
    assert q.shape == (rows, cols) and s.shape == (rows, nb), (what, q.shape, s.shape)
    pad = nb * 128 - cols
    P = torch.nn.functional.pad(X, (0, pad)).view(rows, nb, 128)
    T = torch.nn.functional.pad(tol, (0, pad)).view(rows, nb, 128)
    V = torch.nn.functional.pad(q, (0, pad)).view(rows, nb, 128)
    amax, worst = P.abs().amax(2), T.amax(2)
    if pow2:
        m, e = torch.frexp(s)
        assert bool((m == 0.5).all()), (what, "a scale is no power of two")
        assert bool((448 * s >= (amax - worst) * (1 - 2 * U)).all()), (what, "scale too small")
        assert bool(((448 * s / 2 < (amax + worst) * (1 + 2 * U)) | (s == 2.0 ** -127)).all()), (what, "scale too large")
    else:
        # one division: half a step of FP32, or of its subnormals (2^-150)
        off = (s * 448 - amax).abs() - (worst + amax * 2 * U + 448 * 2.0 ** -150)
        assert bool((off <= 0).all()), (what, "scale", float((off / (amax + 1e-300)).max()))
    zero = s == 0
    assert bool((V[zero.unsqueeze(2).expand_as(V)] == 0).all()), (what, "codes of a zero block")
    S = torch.where(zero, torch.ones_like(s), s).unsqueeze(2)
    y = (P / S).clamp(-448, 448)
    # the value's own tolerance, and two roundings of the FP32 quotient
    d = T / S + 4 * U * y.abs()
    off = (V - y).abs() - (half_step(y.abs() + d) + d)
    off = torch.where(zero.unsqueeze(2), torch.full_like(off, -1.0), off)
    assert bool((off <= 0).all()), (what, "codes", np.unravel_index(int(off.argmax()), off.shape), float(off.max()))


def check_dual(X, tol, q_row, s_row, q_tok, s_tok, what, transpose_out=True, pow2=False):
    check_blocks(X, tol, q_row, s_row, what + " rows", pow2)
    if not transpose_out:
        q_tok, s_tok = q_tok.t(), s_tok.t()
    check_blocks(X.t(), tol.t(), q_tok, s_tok, what + " tokens", pow2)


def norm(z, w, eps):
    """(n, tolerance of n, rstd, relative tolerance of rstd) for float64 z [t][c], w [c]."""
    t, c = z.shape
    r = 1.0 / torch.sqrt((z * z).sum(1) / c + eps)
    # the sum's chain reaches r halved (square root); mean, + eps, sqrt (2 steps), 1 / x
    rel = (chain(c) / 2 + 6) * U
    n = z * r[:, None] * w
    return n, n.abs() * (rel + 3 * U) + 2.0 ** -148, r, rel


def norm_bwd(dy, z, r, w, dres):
    """(dx, tolerance of dx, dw, tolerance of dw), everything float64; r is the FP32 rstd given."""
    t, c = z.shape
    xh, g = z * r[:, None], dy * w
    m = (g * xh).mean(1, keepdim=True)
    mabs = (g * xh).abs().mean(1, keepdim=True)
    dx = r[:, None] * (g - xh * m)
    # m's sum, its product and quotient; then xh m (2 roundings), the difference, the product with r
    tol = r[:, None] * (xh.abs() * (mabs * (chain(c) + 6) * U + 3 * U * m.abs()) + 3 * U * g.abs()) + 3 * U * dx.abs()
    if dres is not None:
        dx = dx + dres
        tol = tol + U * dx.abs()
    # every term of dw passes its thread's 4 tokens, 2 exchanges, 8 waves, then the token tiles in order
    dw = (dy * xh).sum(0)
    dtol = (dy * xh).abs().sum(0) * (4 + 2 + 8 + (t + 127) // 128 + 3) * U
    return dx, tol + 2.0 ** -147, dw, dtol + 2.0 ** -147


def swiglu_bwd(dh, g, u):
    """(dgate, dup, their tolerances), float64."""
    sg, ns = torch.sigmoid(g), torch.sigmoid(-g)
    dup, dgate = dh * g * sg, dh * u * sg * (1 + g * ns)
    # e^-|g| within 2 steps, 1 + e, the reciprocal (1 step) and the products: at most 10 roundings of
    # what enters; 1 + g ns may cancel, so its own error is taken on 1 + |g ns|.  e^-|g| below FP32's
    # normal range (|g| > 87.3) keeps its absolute error of 2^-149.
    tu = 16 * U * dup.abs() + 2.0 ** -148 * (dh * g).abs() + 2.0 ** -148
    mag = (dh * u).abs()
    tg = 16 * U * mag * sg * (1 + (g * ns).abs()) + 2.0 ** -148 * mag * (1 + g.abs()) + 2.0 ** -148
    return dgate, dup, tg, tu


def close_bf16(got, want, tol, what):
    """A BF16 result: one rounding (half a step, 2^-8 of the value; subnormal spacing 2^-133) past tol."""
    off = (f64(got) - want).abs() - (tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -134)
    assert bool((off <= 0).all()), (what, np.unravel_index(int(off.argmax()), off.shape), float(off.max()))


def bf16(rows, cols, std, seed, device="cpu", pad=0):
    """Seeded BF16 [rows][cols] with a padded row stride (NaN in the padding)."""
    gen = torch.Generator().manual_seed(seed)
    ld = (cols + 15) // 16 * 16 + pad
    buf = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16)
    buf[:, :cols] = (torch.randn((rows, cols), generator=gen) * std).to(torch.bfloat16)
    return buf.to(device)[:, :cols]
