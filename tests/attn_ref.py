"""64-bit references of the head norm with rotation, of attention and of their gradients, with bounds on
how far the kernels' results may be from them (absolute, per element; counted roundings).

U is half a step of FP32 and B half a step of BF16, both relative.  A matrix-core product of n terms is
allowed 2 n U of its terms' magnitudes (one rounding or truncation a term).  An
exponential below FP32's normal range (2^-126) is zero, and so may a product or a
BF16 operand below it be: P and dS have that absolute error beside their relative one.
"""
import torch

U, B, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126


def f64(t):
    return t.detach().double().cpu()


# ------------------------------------------------------------------ head norm and rotation

def pairs(dim, rotary, interleaved):
    """Column indices of the pairs' first and second members."""
    j = torch.arange(rotary // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)


def angles(pos, freq, m):
    a = torch.outer(pos.double(), freq.double())
    # the angle's own error, cos and sin (4 steps), the product with m
    err = torch.where(a.abs() < 2.0 ** 20, 2.0 ** -31, 2.0 ** -20) + 10 * U
    return torch.cos(a) * m, torch.sin(a) * m, err * abs(m)


def turn(v, pos, freq, m, interleaved, back=False):
    """v [T][heads][dim] with its pairs turned (back: by the transpose), and the turn's own error bound."""
    first, second = pairs(v.shape[2], 2 * len(freq), interleaved)
    cos, sin, err = (t[:, None] for t in angles(pos, freq, m))
    if back:
        sin = -sin
    a, b = v[..., first], v[..., second]
    out, tol = v.clone(), torch.zeros_like(v)
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    mag = (a.abs() + b.abs()) * (err + 3 * U * abs(m))
    tol[..., first], tol[..., second] = mag, mag
    return out, tol


CHAIN = 8 + 4      # additions a term of a head's sum goes through: a lane's eight, four exchanges


def rope(x, w, eps, pos, freq, m, interleaved):
    """(y, tolerance, rstd, its relative tolerance); x float64 [T][heads][dim]."""
    n, rel, r = x, 0.0, None
    if w is not None:
        r = 1.0 / torch.sqrt((x * x).mean(2) + eps)
        rel = (CHAIN / 2 + 6) * U
        n = x * r[..., None] * w
        rel_n = rel + 3 * U
    else:
        rel_n = 0.0
    y, tol = turn(n, pos, freq, m, interleaved)
    spread, _ = turn(n.abs(), pos, freq, 1.0, interleaved)
    first, second = pairs(x.shape[2], 2 * len(freq), interleaved)
    grow = n.abs() * rel_n
    both = (n[..., first].abs() + n[..., second].abs()) * rel_n * abs(m)
    grow[..., first], grow[..., second] = both, both
    del spread
    return y, tol * (1 + rel_n) + grow, r, rel


def rope_bwd(dy, x, r, w, pos, freq, m, interleaved):
    """(dx, tolerance, dw, tolerance) of one of q and k; r the FP32 rstd given, float64 everything."""
    g, gt = turn(dy, pos, freq, m, interleaved, back=True)
    if w is None:
        return g, gt, None, None
    d = x.shape[2]
    xh, wg, r = x * r[..., None], g * w, r[..., None]
    wgt = gt * w.abs() + 2 * U * wg.abs()
    mean = (wg * xh).mean(2, keepdim=True)
    terms = ((wgt + (CHAIN + 4) * U * wg.abs()) * xh.abs()).mean(2, keepdim=True)
    dx = r * (wg - xh * mean)
    tol = r * (wgt + xh.abs() * (terms + 4 * U * mean.abs()) + 2 * U * wg.abs()) + 3 * U * dx.abs()
    dw = (g * xh).sum((0, 1))
    n = x.shape[0] * x.shape[1]
    # a term: 4 tokens of a thread, 2 exchanges, 8 waves, then every 16th of the tiles and heads, 4 halvings
    steps = 4 + 2 + 8 + -(-n // (128 * 16)) + x.shape[1] + 4
    dwt = ((gt + (steps + 2) * U * g.abs()) * xh.abs()).sum((0, 1))
    assert d in (64, 128)
    return dx, tol, dw, dwt


# ------------------------------------------------------------------ attention

def hidden(n, m, causal):
    if not causal:
        return torch.zeros((n, m), dtype=torch.bool)
    return torch.ones((n, m), dtype=torch.bool).triu(m - n + 1)


def head(q, k, v, scale, causal):
    """One head of one sequence, float64: (o, tolerance of o before its rounding, lse, its tolerance, P, dS-free
    score error per row)."""
    n, m, d = q.shape[0], k.shape[0], q.shape[1]
    if m == 0 or n == 0:
        z = torch.zeros((n, d), dtype=torch.float64)
        e = torch.zeros((n, 1), dtype=torch.float64)
        return z, z, torch.full((n,), -torch.inf, dtype=torch.float64), e[:, 0], torch.zeros((n, m), dtype=torch.float64), e
    s = scale * (q @ k.t())
    hide = hidden(n, m, causal)
    mag = scale * (q.abs() @ k.abs().t())
    s = s.masked_fill(hide, -torch.inf)
    lse = torch.logsumexp(s, 1)
    seen = ~torch.isinf(lse)
    p = torch.where(hide, 0.0, torch.exp(s - torch.where(seen, lse, torch.zeros_like(lse))[:, None]))
    # scores: the product, the scale's and the maximum's roundings; the exponential's one step
    top = torch.where(hide, 0.0, mag).amax(1, keepdim=True)
    es = top * (2 * d + 8) * U + 4 * U
    o = p @ v
    acc = (m + 16) * 2 * U
    # P is formed relative to a running maximum at most 2^8 below the row's: TINY there is 2^8 TINY of a sum of
    # 2^-8 or more
    tol = (B + 2 * es + acc) * (p @ v.abs()) + 2.0 ** 16 * TINY * v.abs().sum(0)
    lt = es[:, 0] + acc + 4 * U * torch.where(seen, lse, 0.0).abs() + 4 * U * top[:, 0]
    return o, tol, lse, lt, p, es


def head_bwd(q, k, v, do, o, lse, scale, causal):
    """Gradients of one head, float64, with the forward's o and lse as given: (dq, dk, dv, their tolerances)."""
    n, m, d = q.shape[0], k.shape[0], q.shape[1]
    if m == 0 or n == 0:
        zq, zk = torch.zeros((n, d), dtype=torch.float64), torch.zeros((m, d), dtype=torch.float64)
        return zq, zk, zk, zq, zk, zk
    hide = hidden(n, m, causal)
    seen = ~torch.isinf(lse)
    base = torch.where(seen, lse, torch.zeros_like(lse))[:, None]
    p = torch.where(hide, 0.0, torch.exp(scale * (q @ k.t()) - base))
    top = torch.where(hide, 0.0, scale * (q.abs() @ k.abs().t())).amax(1, keepdim=True)
    ep = (2 * d + 8) * U * (top + base.abs()) + 8 * U
    dp, dd = do @ v.t(), (do * o).sum(1, keepdim=True)
    edd = 2 * d * U * (do * o).abs().sum(1, keepdim=True)
    # rows that see at most 32 keys: D from P dP itself, 32 more additions and P's own error
    few = (~hide).sum(1, keepdim=True) <= 32
    own = (p * dp).sum(1, keepdim=True)
    eown = (p * (2 * (d + 40) * U + ep) * (do.abs() @ v.abs().t())).sum(1, keepdim=True)
    dd, edd = torch.where(few, own, dd), torch.where(few, eown, edd)
    edp = 2 * d * U * (do.abs() @ v.abs().t() + dd.abs()) + edd
    ds = p * (dp - dd)
    eds = ds.abs() * (B + ep + 4 * U) + p * edp * (1 + B) + TINY * (1 + (dp - dd).abs() + edp)
    aq, ak = (m + 16) * 2 * U, (n + 16) * 2 * U
    dq, dk, dv = scale * ds @ k, scale * ds.t() @ q, p.t() @ do
    tq = scale * (eds + aq * ds.abs()) @ k.abs()
    tk = scale * (eds + ak * ds.abs()).t() @ q.abs()
    tv = (p * (B + ep + 4 * U + ak) + TINY).t() @ do.abs()
    return dq, dk, dv, tq, tk, tv


def heads(t, rows, h, dim):
    return t[rows, h * dim:(h + 1) * dim]


def spans(offsets, lengths):
    """Row slices of the sequences."""
    if lengths is None:
        return [slice(a, b) for a, b in zip(offsets, offsets[1:])]
    return [slice(a, a + n) for a, n in zip(offsets, lengths)]


def attention(q, k, v, dim, qs, ks, scale, causal):
    """(o, tolerance, lse, tolerance) over all sequences; NaN in rows of no sequence."""
    q, k, v = f64(q), f64(k), f64(v)
    hq, hk = q.shape[1] // dim, k.shape[1] // dim
    o, ot = torch.full_like(q, float("nan")), torch.zeros_like(q)
    lse = torch.full((hq, q.shape[0]), float("nan"), dtype=torch.float64)
    lt = torch.zeros_like(lse)
    for a, b in zip(qs, ks):
        for h in range(hq):
            g = h // (hq // hk)
            r = head(heads(q, a, h, dim), heads(k, b, g, dim), heads(v, b, g, dim), scale, causal)
            o[a, h * dim:(h + 1) * dim], ot[a, h * dim:(h + 1) * dim], lse[h, a], lt[h, a] = r[:4]
    return o, ot, lse, lt


def attention_bwd(do, q, k, v, o, lse, dim, qs, ks, scale, causal):
    """((dq, tolerance), (dk, ..), (dv, ..)); NaN in rows of no sequence."""
    do, q, k, v, o, lse = (f64(t) for t in (do, q, k, v, o, lse))
    hq, hk = q.shape[1] // dim, k.shape[1] // dim
    res = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    tol = [torch.zeros_like(t) for t in (q, k, v)]
    for a, b in zip(qs, ks):
        for t in res[1:]:
            t[b] = 0.0
        for h in range(hq):
            g = h // (hq // hk)
            r = head_bwd(heads(q, a, h, dim), heads(k, b, g, dim), heads(v, b, g, dim), heads(do, a, h, dim),
                         heads(o, a, h, dim), lse[h, a], scale, causal)
            cq, ck = slice(h * dim, (h + 1) * dim), slice(g * dim, (g + 1) * dim)
            res[0][a, cq], tol[0][a, cq] = r[0], r[3]
            for i in (1, 2):
                res[i][b, ck] += r[i]
                tol[i][b, ck] += r[i + 3]
    return list(zip(res, tol))


def close_bf16(got, want, tol, what):
    """BF16 results: half a step of BF16 past tol where want is a number, the old contents (a NaN) where not."""
    got = f64(got)
    free = torch.isnan(want)
    assert bool(torch.isnan(got[free]).all()), (what, "rows of no sequence were written")
    off = (got - want).abs() - (tol + B * (want.abs() + tol) + 2.0 ** -134)
    off = torch.where(free, torch.full_like(off, -1.0), off)
    assert bool((off <= 0).all()), (what, [int(i) for i in torch.unravel_index(torch.nan_to_num(off, nan=1e30).argmax(),
                                                                               off.shape)], float(off.max()))
    # rounding errors of many terms average out: the whole result is off by less than one half step of P
    # (2^-8, uniform: / sqrt 3) and one of the result, together 0.82 of 2^-8
    w, g = want[~free], got[~free]
    if w.numel() > 4096 and float(w.norm()) > 0:
        assert float((g - w).norm() / w.norm()) <= B, (what, "relative error", float((g - w).norm() / w.norm()))


def bf16(gen, rows, cols, std=1.0, pad=0, dev="cpu"):
    """Seeded BF16 [rows][cols] with a padded row stride and NaN in the padding."""
    ld = (cols + 15) // 16 * 16 + pad
    buf = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16)
    buf[:, :cols] = (torch.randn((rows, cols), generator=gen) * std).to(torch.bfloat16)
    return buf.to(dev)[:, :cols]


def i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out
