"""puro_fp8_qk_norm_rope and its gradient against the 64-bit definition."""
import math

import pytest
import torch

import blockwise_fp8_gemm_amd as pf
import attn_ref as ref
from fused_ref import check_dual

pytestmark = pytest.mark.gpu

EPS = 1e-6


def case(dev, tokens, hq, hk, dim, rotary, norm, wdt=torch.float32, seed=0, pad=0, positions=None, base=1e4, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    c = {"q": ref.bf16(gen, tokens, hq * dim, std, pad, dev), "k": ref.bf16(gen, tokens, hk * dim, std, 2 * pad, dev)}
    if tokens > 2:
        c["k"][1] = 0.0       # a head of zeros
    if positions is None:
        positions = torch.randint(0, 5000, (tokens,), generator=gen)
    c["pos"] = torch.as_tensor(positions).to(torch.int32).to(dev)
    c["freq"] = (base ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))).float().to(dev) if rotary else None
    c["wq"] = (1 + 0.2 * torch.randn((dim,), generator=gen)).to(wdt).to(dev) if norm else None
    c["wk"] = (1 + 0.2 * torch.randn((dim,), generator=gen)).to(wdt).to(dev) if norm else None
    for name, h in (("dq", hq), ("dk", hk), ("dv", hk)):
        c[name] = ref.bf16(gen, tokens, h * dim, 1e-3, pad, dev)
    return c


def angles(c):
    return ref.f64(c["pos"]), ref.f64(c["freq"]) if c["freq"] is not None else torch.zeros((0,), dtype=torch.float64)


def opt64(t):
    return None if t is None else ref.f64(t)


def forward(dev, tokens, hq, hk, dim, rotary, norm, interleaved, m=1.0, **kw):
    c = case(dev, tokens, hq, hk, dim, rotary, norm, **kw)
    y = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], dim, c["pos"], c["freq"], c["wq"], c["wk"], EPS, m, interleaved)
    torch.cuda.synchronize()
    pos, freq = angles(c)
    rs = []
    for got, x, w, what in ((y[0], c["q"], c["wq"], "q"), (y[1], c["k"], c["wk"], "k")):
        want, tol, r, rel = ref.rope(ref.f64(x).view(tokens, x.shape[1] // dim, dim), opt64(w), EPS, pos, freq, m, interleaved)
        ref.close_bf16(got, want.flatten(1), tol.flatten(1), (what, tokens, hq, hk, dim, rotary, norm, interleaved))
        rs.append((r, rel))
    if norm:
        want = torch.cat((rs[0][0], rs[1][0]), 1)
        assert bool(((ref.f64(y[2]) - want).abs() <= rs[0][1] * want).all())
    else:
        assert y[2] is None


@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 32), (64, 16), (64, 0), (128, 128), (128, 64), (128, 48), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_forward(dev, dim, rotary, interleaved, norm):
    forward(dev, 37, 4, 2, dim, rotary, norm, interleaved, m=1.0 if rotary % 32 else 1.3, seed=rotary, pad=16)


@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (1, 16, 8), (2, 3, 5), (5, 40, 40), (129, 7, 1), (700, 16, 8), (5000, 2, 1),
                                          (0, 2, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_forward_sizes(dev, tokens, hq, hk, dim):
    forward(dev, tokens, hq, hk, dim, dim, True, False, wdt=torch.bfloat16, seed=tokens)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(dev, interleaved):
    """Angles of positions up to the largest, negative ones, and frequencies above one."""
    pos = [0, 1, -1, 2 ** 20, 2 ** 20 - 1, 10 ** 7, 2 ** 31 - 1, -2 ** 31, 123456789]
    forward(dev, len(pos), 2, 1, 128, 128, False, interleaved, positions=pos, base=1e6)


def test_scaled_frequencies(dev):
    """Positions of a longer context by changed frequencies and a scale: the call of the changed formula."""
    c = case(dev, 50, 2, 1, 64, 64, True, seed=4, positions=torch.arange(50) * 4000)
    freq = c["freq"] / torch.linspace(1.0, 8.0, 32, device=dev)
    m = 0.1 * math.log(8.0) + 1.0
    y, _, _ = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], 64, c["pos"], freq, c["wq"], c["wk"], EPS, m)
    want, tol, _, _ = ref.rope(ref.f64(c["q"]).view(50, 2, 64), ref.f64(c["wq"]), EPS, ref.f64(c["pos"]), ref.f64(freq), m, False)
    ref.close_bf16(y, want.flatten(1), tol.flatten(1), "scaled")


@pytest.mark.parametrize("dim,tokens", [(64, 300), (128, 300), (128, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(dev, dim, tokens, interleaved):
    c = case(dev, tokens, 6, 3, dim, dim // 2, True, seed=5, pad=16)
    args = (dim, c["pos"], c["freq"], c["wq"], c["wk"], EPS, 1.0, interleaved)
    want = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], *args)
    got = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], *args, q_out=c["q"], k_out=c["k"], store_rstd=False)
    assert got[0].data_ptr() == c["q"].data_ptr() and got[2] is None
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def backward(dev, tokens, hq, hk, dim, rotary, norm, interleaved, m=1.0, transpose_out=True, pow2=False, store_dx=True, **kw):
    c = case(dev, tokens, hq, hk, dim, rotary, norm, **kw)
    H = hq + hk
    rstd = None
    if norm:
        x = torch.cat((ref.f64(c["q"]), ref.f64(c["k"])), 1).view(tokens, H, dim)
        rstd = (1.0 / torch.sqrt(x.square().mean(2) + EPS)).float().to(dev)
    got = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(
        c["dq"], c["dk"], c["dv"], c["q"] if norm else None, c["k"] if norm else None, dim, c["pos"], c["freq"], rstd=rstd,
        q_weight=c["wq"], k_weight=c["wk"], rope_scale=m, interleaved=interleaved, transpose_out=transpose_out,
        store_dx=store_dx, pow2=pow2)
    torch.cuda.synchronize()
    dx, dwq, dwk, *codes = got
    pos, freq = angles(c)
    parts, tols = [], []
    for dy, x, w, hs, dw, what in ((c["dq"], c["q"], c["wq"], slice(0, hq), dwq, "dwq"),
                                   (c["dk"], c["k"], c["wk"], slice(hq, H), dwk, "dwk")):
        r = ref.f64(rstd)[:, hs] if norm else None
        want, tol, wdw, tdw = ref.rope_bwd(ref.f64(dy).view(tokens, dy.shape[1] // dim, dim), ref.f64(x).view(tokens, x.shape[1] // dim, dim), r, opt64(w),
                                           pos, freq, m, interleaved)
        parts.append(want.flatten(1))
        tols.append(tol.flatten(1))
        if norm:
            off = (ref.f64(dw) - wdw).abs() - tdw - 2.0 ** -147
            assert bool((off <= 0).all()), (what, float(off.max()))
        else:
            assert dw is None
    dv = ref.f64(c["dv"])
    want, tol = torch.cat((*parts, dv), 1), torch.cat((*tols, torch.zeros_like(dv)), 1) + 2.0 ** -147
    what = (tokens, hq, hk, dim, rotary, norm, interleaved)
    if store_dx:
        ref.close_bf16(dx, want, tol, what)
    else:
        assert dx is None
    check_dual(want, tol, *codes, str(what), transpose_out, pow2)


@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 32), (64, 0), (128, 128), (128, 64), (128, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_backward(dev, dim, rotary, interleaved, norm):
    backward(dev, 131, 4, 2, dim, rotary, norm, interleaved, m=1.0 if rotary % 32 else 1.3, seed=rotary, pad=16)


@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (1, 16, 8), (127, 3, 5), (128, 2, 1), (257, 7, 1), (700, 16, 8), (3000, 2, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_backward_sizes(dev, tokens, hq, hk, dim):
    """Odd head counts put two kinds of heads, or the tensor's end, inside a block of 64-wide heads."""
    backward(dev, tokens, hq, hk, dim, dim, True, False, wdt=torch.bfloat16, seed=tokens)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("transpose_out", [True, False])
@pytest.mark.parametrize("pow2", [True, False])
def test_backward_layouts(dev, dim, transpose_out, pow2):
    backward(dev, 200, 5, 2, dim, dim, True, True, transpose_out=transpose_out, pow2=pow2, store_dx=False, seed=6)


def test_backward_accumulates(dev):
    c = case(dev, 300, 4, 2, 64, 64, True, seed=8)
    _, _, rstd = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], 64, c["pos"], c["freq"], c["wq"], c["wk"], EPS)
    args, kw = (c["dq"], c["dk"], c["dv"], c["q"], c["k"], 64, c["pos"], c["freq"], rstd, c["wq"], c["wk"]), {}
    _, dwq, dwk, *codes = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(*args)
    old = torch.randn((2, 64), generator=torch.Generator().manual_seed(1)).to(dev)
    a, b = old[0].clone(), old[1].clone()
    _, x, y, *again = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(*args, dwq=a, dwk=b, accumulate=True, **kw)
    assert torch.equal(x, old[0] + dwq) and torch.equal(y, old[1] + dwk)
    assert all(torch.equal(p, q) for p, q in zip(codes, again))
    # no tokens: the weights' gradients are zero, or stay
    empty = {n: c[n][:0] for n in ("dq", "dk", "dv", "q", "k")}
    none = (empty["dq"], empty["dk"], empty["dv"], empty["q"], empty["k"], 64, c["pos"][:0], c["freq"], rstd[:0], c["wq"], c["wk"])
    _, x, y, *_ = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(*none)
    assert not x.any() and not y.any()
    _, x, _, *_ = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(*none, dwq=a, dwk=b, accumulate=True)
    assert torch.equal(x, old[0] + dwq)


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_against_differences(dev, interleaved):
    """d/dt of sum dq y(q + t x) + ... by central differences of the 64-bit forward."""
    t, hq, hk, dim = 40, 3, 2, 64
    c = case(dev, t, hq, hk, dim, 32, True, seed=9)
    m = 1.1
    _, _, rstd = pf.puro_fp8_qk_norm_rope(c["q"], c["k"], dim, c["pos"], c["freq"], c["wq"], c["wk"], EPS, m, interleaved)
    dx, dwq, dwk, *_ = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(
        c["dq"], c["dk"], c["dv"], c["q"], c["k"], dim, c["pos"], c["freq"], rstd, c["wq"], c["wk"], m, interleaved, store_dx=True)
    pos, freq = angles(c)
    gen = torch.Generator().manual_seed(10)
    dx = ref.f64(dx)
    for x, w, dy, cols, dw in ((c["q"], c["wq"], c["dq"], slice(0, hq * dim), dwq),
                               (c["k"], c["wk"], c["dk"], slice(hq * dim, (hq + hk) * dim), dwk)):
        x, w, dy = ref.f64(x).view(t, -1, dim), ref.f64(w), ref.f64(dy).view(t, -1, dim)
        a, b = torch.randn(x.shape, generator=gen, dtype=torch.float64), torch.randn(w.shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        keep = x.abs().amax((0, 2)) > 0
        a *= (x.abs().amax(2) > 0)[..., None]      # a head of zeros sits where the norm bends: not moved
        loss = lambda x, w: float((dy * ref.rope(x, w, EPS, pos, freq, m, interleaved)[0]).sum())  # noqa: E731
        slope = (loss(x + h * a, w) - loss(x - h * a, w)) / (2 * h)
        g = dx[:, cols].view(t, -1, dim)
        assert abs(float((g * a).sum()) - slope) <= float((ref.B * 1.1 * g.abs() * a.abs()).sum()) + 1e-7
        slope = (loss(x, w + h * b) - loss(x, w - h * b)) / (2 * h)
        assert abs(float((ref.f64(dw) * b).sum()) - slope) <= 1e-5 * float((ref.f64(dw) * b).abs().sum()) + 1e-7
        assert bool(keep.all())
