"""The attention and head-norm entry points on the host: bad arguments are refused before any launch, through the
C ABI and the binding; the 64-bit references against each other."""
import ctypes

import pytest
import torch

import attn_ref as ref
import blockwise_fp8_gemm_amd as pf

OK, NULL, SHAPE, ALIGN, ENUM, WORKSPACE, VALUE = 0, 1, 2, 3, 4, 5, 8
PTR = 1 << 20               # aligned, never dereferenced (validation fails first)
P, NUL = ctypes.c_void_p(PTR), ctypes.c_void_p(0)
ODD, TWO = ctypes.c_void_p(PTR + 4), ctypes.c_void_p(PTR + 2)
BIG = (1 << 23) + 1


def rope(**kw):
    d = dict(heads_q=4, heads_kv=2, head_dim=64, rotary_dim=64, interleaved=0, tokens=8, positions=PTR, inv_freq=PTR,
             rope_scale=1.0, wq=PTR, wk=PTR, wdt=0, eps=1e-6)
    d.update(kw)
    return pf.QkNormRope(**d)


ROPE_BAD = [(dict(heads_q=0), SHAPE), (dict(heads_kv=0), SHAPE), (dict(heads_q=1025), SHAPE), (dict(heads_kv=1025), SHAPE),
            (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(rotary_dim=-16), SHAPE), (dict(rotary_dim=80), SHAPE),
            (dict(rotary_dim=24), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=BIG), SHAPE), (dict(interleaved=2), ENUM),
            (dict(wdt=2), ENUM), (dict(positions=0), NULL), (dict(inv_freq=0), NULL), (dict(wk=0), NULL), (dict(wq=0), NULL),
            (dict(wq=PTR + 4), ALIGN), (dict(positions=PTR + 2), ALIGN), (dict(inv_freq=PTR + 1), ALIGN),
            (dict(eps=0.0), VALUE), (dict(eps=float("inf")), VALUE), (dict(eps=1e-39), VALUE),
            (dict(rope_scale=float("nan")), VALUE), (dict(rope_scale=float("inf")), VALUE)]


def _rope_fwd(shape=None, q=P, ldq=256, k=P, ldk=128, qo=P, ldqo=256, ko=P, ldko=128, rstd=NUL):
    return pf.lib().puro_fp8_qk_norm_rope(shape if shape is not None else rope(), q, ldq, k, ldk, qo, ldqo, ko, ldko, rstd, None)


def _rope_bwd(shape=None, suffix="", dq=P, lddq=256, dk=P, lddk=128, dv=P, lddv=128, q=P, ldq=256, k=P, ldk=128, rstd=P,
              dx=NUL, lddx=0, dwq=P, dwk=P, acc=0, qr=P, ldqr=512, sr=P, t=1, qt=P, ldqt=16, st=P, ws=P, n=1 << 24):
    return getattr(pf.lib(), "puro_fp8_qk_norm_rope_bwd_quant_dual" + suffix)(
        shape if shape is not None else rope(), dq, lddq, dk, lddk, dv, lddv, q, ldq, k, ldk, rstd, dx, lddx, dwq, dwk, acc,
        qr, ldqr, sr, t, qt, ldqt, st, ws, n, None)


@pytest.mark.parametrize("fields,status", ROPE_BAD)
def test_rope_shapes(fields, status):
    assert _rope_fwd(rope(**fields)) == status
    assert _rope_bwd(rope(**fields)) == status


def test_rope_refusals():
    assert pf.lib().puro_fp8_qk_norm_rope(None, P, 256, P, 128, P, 256, P, 128, NUL, None) == NULL
    for name in ("q", "k", "qo", "ko"):
        assert _rope_fwd(**{name: NUL}) == NULL and _rope_fwd(**{name: ODD}) == ALIGN, name
    for name, low, odd in (("ldq", 240, 264), ("ldk", 112, 136), ("ldqo", 240, 264), ("ldko", 112, 136)):
        assert _rope_fwd(**{name: low}) == SHAPE and _rope_fwd(**{name: odd}) == ALIGN, name
    assert _rope_fwd(rstd=TWO) == ALIGN
    assert _rope_fwd(rope(tokens=0, positions=0, inv_freq=0), q=NUL, k=NUL, qo=NUL, ko=NUL) == OK


@pytest.mark.parametrize("suffix", ["", "_pow2"])
def test_rope_bwd_refusals(suffix):
    def call(**kw):
        return _rope_bwd(suffix=suffix, **kw)
    assert call(t=2) == ENUM and call(acc=2) == ENUM
    for name in ("dq", "dk", "dv", "q", "k", "qr", "sr", "qt", "st", "rstd", "dwq", "dwk"):
        assert call(**{name: NUL}) == NULL, name
    for name in ("dq", "dk", "dv", "q", "k", "qr", "qt"):
        assert call(**{name: ODD}) == ALIGN, name
    for name, low, odd in (("lddq", 240, 264), ("lddk", 112, 136), ("lddv", 112, 136), ("ldq", 240, 264), ("ldk", 112, 136),
                           ("ldqr", 496, 520), ("ldqt", 0, 24)):
        assert call(**{name: low}) == SHAPE and call(**{name: odd}) == ALIGN, name
    assert call(dx=P, lddx=496) == SHAPE and call(dx=P, lddx=520) == ALIGN and call(dx=ODD, lddx=512) == ALIGN
    for name in ("rstd", "dwq", "dwk"):
        assert call(**{name: TWO}) == ALIGN, name
    need = pf.lib().puro_fp8_qk_norm_rope_bwd_workspace_size(rope())
    assert need > 0 and call(n=need - 1) == WORKSPACE and call(ws=NUL) == WORKSPACE and call(ws=ODD) == WORKSPACE
    for fields, status in ROPE_BAD:
        if status == SHAPE:
            assert pf.lib().puro_fp8_qk_norm_rope_bwd_workspace_size(rope(**fields)) == 0
    assert pf.lib().puro_fp8_qk_norm_rope_bwd_workspace_size(None) == 0
    # without weights and tokens there is nothing to write
    none = rope(tokens=0, wq=0, wk=0, positions=0, inv_freq=0)
    assert call(shape=none, dq=NUL, dk=NUL, dv=NUL, q=NUL, k=NUL, rstd=NUL, dwq=NUL, dwk=NUL, qr=NUL, sr=NUL, qt=NUL, st=NUL,
                ws=NUL, n=0) == OK


def attn(**kw):
    d = dict(heads_q=4, heads_kv=2, head_dim=64, sequences=2, causal=1, tokens_q=64, tokens_k=96, max_q=40, max_k=96,
             q_offsets=PTR, q_lengths=0, k_offsets=PTR, k_lengths=0, scale=0.125)
    d.update(kw)
    return pf.Attention(**d)


ATTN_BAD = [(dict(heads_q=0), SHAPE), (dict(heads_kv=0), SHAPE), (dict(heads_q=5), SHAPE), (dict(heads_q=1026), SHAPE),
            (dict(head_dim=32), SHAPE), (dict(head_dim=256), SHAPE), (dict(sequences=-1), SHAPE), (dict(tokens_q=-1), SHAPE),
            (dict(tokens_k=BIG), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_k=BIG), SHAPE), (dict(causal=2), ENUM),
            (dict(causal=-1), ENUM), (dict(q_offsets=0), NULL), (dict(k_offsets=0), NULL), (dict(q_offsets=PTR + 2), ALIGN),
            (dict(k_offsets=PTR + 1), ALIGN), (dict(q_lengths=PTR + 2), ALIGN), (dict(k_lengths=PTR + 2), ALIGN),
            (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=float("nan")), VALUE),
            (dict(scale=float("inf")), VALUE), (dict(scale=2.0 ** -65), VALUE), (dict(scale=2.0 ** 65), VALUE),
            # more work items than a grid has
            (dict(sequences=2 ** 31 - 1, tokens_q=2 ** 23, tokens_k=2 ** 23, max_q=2 ** 23, max_k=2 ** 23), SHAPE),
            (dict(heads_q=1024, heads_kv=1, tokens_q=2 ** 23, max_q=2 ** 23), SHAPE),
            (dict(sequences=2 ** 31 - 1, max_q=1, max_k=1), SHAPE)]

# the most that is promised: sequences x heads_kv x ceil(n / 64) just below 2^23
ATTN_MANY = [dict(sequences=2 ** 14 - 1, heads_q=8, heads_kv=8, max_q=4096), dict(sequences=2 ** 14 - 1, heads_q=1, heads_kv=1, max_q=2 ** 15),
             dict(sequences=2 ** 22 - 1, heads_q=4, heads_kv=2, max_q=1), dict(sequences=2 ** 14 - 1, heads_q=64, heads_kv=8, max_q=512),
             dict(sequences=1, heads_q=127, heads_kv=127, max_q=2 ** 22), dict(sequences=2 ** 21 - 1, heads_q=20, heads_kv=4, max_q=12),
             dict(sequences=1, heads_q=128, heads_kv=1, max_q=2 ** 22), dict(sequences=63, heads_q=1, heads_kv=1, max_q=2 ** 23)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [2 ** 23, 1 << 16])
@pytest.mark.parametrize("fields", ATTN_MANY)
def test_attention_sizes_that_are_promised(fields, tokens, dim):
    for max_k in (64, 64 * (fields["max_q"] * (fields["heads_q"] // fields["heads_kv"]) // 64)):
        shape = attn(tokens_q=tokens, tokens_k=tokens, head_dim=dim, **dict(fields, max_k=min(max_k, 2 ** 23)))
        assert pf.lib().puro_fp8_attention_bwd_workspace_size(shape) > 0
        # one that fits is told from one that does not by the check that comes next
        assert _fwd(shape, ldq=2 ** 22, ldk=2 ** 22, ldv=2 ** 22, ldo=2 ** 22, lse=TWO) == ALIGN


def _fwd(shape=None, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, o=P, ldo=256, lse=P, ws=NUL, n=0):
    return pf.lib().puro_fp8_attention(shape if shape is not None else attn(), q, ldq, k, ldk, v, ldv, o, ldo, lse, ws, n, None)


def _bwd(shape=None, do=P, lddo=256, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, o=P, ldo=256, lse=P, dq=P, lddq=256, dk=P,
         lddk=128, dv=P, lddv=128, ws=P, n=1 << 30):
    return pf.lib().puro_fp8_attention_bwd(shape if shape is not None else attn(), do, lddo, q, ldq, k, ldk, v, ldv, o, ldo, lse,
                                           dq, lddq, dk, lddk, dv, lddv, ws, n, None)


@pytest.mark.parametrize("fields,status", ATTN_BAD)
def test_attention_shapes(fields, status):
    assert _fwd(attn(**fields)) == status
    assert _bwd(attn(**fields)) == status
    if status == SHAPE:
        assert pf.lib().puro_fp8_attention_workspace_size(attn(**fields)) == 0
        assert pf.lib().puro_fp8_attention_bwd_workspace_size(attn(**fields)) == 0


def test_attention_refusals():
    L = pf.lib()
    assert L.puro_fp8_attention(None, P, 256, P, 128, P, 128, P, 256, P, NUL, 0, None) == NULL
    assert L.puro_fp8_attention_workspace_size(None) == 0 and L.puro_fp8_attention_bwd_workspace_size(None) == 0
    for call, names in ((_fwd, ("q", "k", "v", "o")), (_bwd, ("do", "q", "k", "v", "o", "dq", "dk", "dv"))):
        for name in names:
            assert call(**{name: NUL}) == NULL and call(**{name: ODD}) == ALIGN, name
            ld = {"do": "lddo", "dq": "lddq", "dk": "lddk", "dv": "lddv"}.get(name, "ld" + name)
            wide = name in ("q", "o", "do", "dq")
            assert call(**{ld: 240 if wide else 112}) == SHAPE and call(**{ld: 264 if wide else 136}) == ALIGN, ld
        assert call(lse=TWO) == ALIGN
    assert _bwd(lse=NUL) == NULL
    need = L.puro_fp8_attention_bwd_workspace_size(attn())
    assert need >= 2 * 4 * 64 * 4 and _bwd(n=need - 1) == WORKSPACE and _bwd(ws=NUL) == WORKSPACE and _bwd(ws=ODD) == WORKSPACE
    # a single token over long keys is split: it needs a workspace
    long = attn(sequences=1, tokens_q=1, max_q=1, tokens_k=100000, max_k=100000)
    need = L.puro_fp8_attention_workspace_size(long)
    assert need > 0 and _fwd(long) == WORKSPACE and _fwd(long, ws=P, n=need - 1) == WORKSPACE and _fwd(long, ws=ODD, n=need) == WORKSPACE
    assert L.puro_fp8_attention_workspace_size(attn()) == 0
    # nothing to write
    assert _fwd(attn(sequences=0, q_offsets=0, k_offsets=0)) == OK
    assert _fwd(attn(tokens_q=0), q=NUL, o=NUL, lse=NUL) == OK and _fwd(attn(max_q=0)) == OK
    assert _bwd(attn(sequences=0, q_offsets=0, k_offsets=0)) == OK


def test_binding_refusals():
    """Shapes, dtypes and missing arguments by name, before a GPU is looked for."""
    def bf(r, c):
        return torch.zeros((r, c), dtype=torch.bfloat16)
    off = torch.zeros((2,), dtype=torch.int32)
    for call in (lambda: pf.puro_fp8_attention(bf(4, 128), bf(4, 64), bf(4, 64), 64, off, off, 4, 4),
                 lambda: pf.puro_fp8_attention_bwd(bf(4, 128), bf(4, 128), bf(4, 64), bf(4, 64), bf(4, 128),
                                                   torch.zeros((2, 4)), 64, off, off, 4, 4),
                 lambda: pf.puro_fp8_attention(q=bf(4, 128), k=bf(4, 64), v=bf(4, 64), head_dim=64, q_offsets=off,
                                               k_offsets=off, max_q=4, max_k=4),
                 lambda: pf.puro_fp8_qk_norm_rope(q=bf(4, 128), k=bf(4, 64), head_dim=64, positions=off, inv_freq=off)):
        with pytest.raises(ValueError, match="on the GPU|positions"):
            call()
    with pytest.raises(ValueError, match="whole heads"):
        pf.puro_fp8_attention(bf(4, 100), bf(4, 64), bf(4, 64), 64, off, off, 4, 4)
    with pytest.raises(ValueError, match="head_dim"):
        pf.puro_fp8_attention(bf(4, 96), bf(4, 96), bf(4, 96), 96, off, off, 4, 4)
    with pytest.raises(ValueError, match="2-D"):
        pf.puro_fp8_attention(torch.zeros((4,), dtype=torch.bfloat16), bf(4, 64), bf(4, 64), 64, off, off, 4, 4)
    with pytest.raises(ValueError, match="head_dim"):
        pf.puro_fp8_qk_norm_rope(bf(4, 96), bf(4, 96), 96)
    with pytest.raises(ValueError, match="both or neither"):
        pf.puro_fp8_qk_norm_rope(bf(4, 128), bf(4, 64), 64, q_weight=torch.ones((64,)))
    with pytest.raises(ValueError, match="positions are needed"):
        pf.puro_fp8_qk_norm_rope(bf(4, 128), bf(4, 64), 64, inv_freq=torch.ones((32,)))


# ------------------------------------------------------------------ the references

def test_reference_forward_against_a_direct_sum():
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, 64), generator=gen, dtype=torch.float64) for n in (5, 9, 9))
    o, _, lse, _, _, _ = ref.head(q, k, v, 0.3, True)
    for i in range(5):
        w = [float(torch.exp(0.3 * (q[i] * k[j]).sum())) for j in range(i + 5)]
        assert abs(float(lse[i]) - float(torch.log(torch.tensor(sum(w), dtype=torch.float64)))) < 1e-12
        want = sum(x * v[j] for j, x in enumerate(w)) / sum(w)
        assert float((o[i] - want).abs().max()) < 1e-12


@pytest.mark.parametrize("causal", [True, False])
def test_reference_gradient_against_autograd(causal):
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((n, 64), generator=gen, dtype=torch.float64, requires_grad=True) for n in (7, 11, 11))
    do = torch.randn((7, 64), generator=gen, dtype=torch.float64)
    s = (0.2 * q @ k.t()).masked_fill(ref.hidden(7, 11, causal), -torch.inf)
    o = torch.softmax(s, 1) @ v
    (o * do).sum().backward()
    got = ref.head_bwd(q.detach(), k.detach(), v.detach(), do, o.detach(), torch.logsumexp(s, 1).detach(), 0.2, causal)
    for g, t in zip(got, (q, k, v)):
        assert float((g - t.grad).abs().max()) < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_keeps_inner_products(interleaved):
    """A rotation by positions leaves q . k a function of their distance."""
    gen = torch.Generator().manual_seed(3)
    q, k = (torch.randn((1, 1, 64), generator=gen, dtype=torch.float64).expand(6, 1, 64) for _ in range(2))
    freq = 1e4 ** (-torch.arange(16, dtype=torch.float64) / 16)
    a = ref.turn(q, torch.tensor([0., 5., 100., 1e6, 7., 9.]), freq, 1.0, interleaved)[0]
    b = ref.turn(k, torch.tensor([3., 8., 103., 1e6 + 3, 10., 12.]), freq, 1.0, interleaved)[0]
    dots = (a * b).sum(2)
    assert float((dots - dots[0]).abs().max()) < 1e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rope_gradient_against_autograd(interleaved):
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((5, 2, 64), generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn((64,), generator=gen, dtype=torch.float64, requires_grad=True)
    dy = torch.randn((5, 2, 64), generator=gen, dtype=torch.float64)
    pos, freq = torch.arange(5.0, dtype=torch.float64) * 31, 1e4 ** (-torch.arange(24, dtype=torch.float64) / 24)
    r = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6)
    n = x * r * w
    first, second = ref.pairs(64, 48, interleaved)
    c, s = torch.cos(torch.outer(pos, freq))[:, None] * 1.2, torch.sin(torch.outer(pos, freq))[:, None] * 1.2
    y = n.index_copy(2, first, n[..., first] * c - n[..., second] * s).index_copy(2, second, n[..., second] * c + n[..., first] * s)
    (y * dy).sum().backward()
    dx, _, dw, _ = ref.rope_bwd(dy, x.detach(), r.detach()[..., 0], w.detach(), pos, freq, 1.2, interleaved)
    assert float((dx - x.grad).abs().max()) < 1e-12 and float((dw - w.grad).abs().max()) < 1e-12
