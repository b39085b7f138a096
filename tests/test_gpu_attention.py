"""puro_fp8_attention against the 64-bit definition: packed, padded and empty sequences, grouped heads, single
tokens and chunks over longer keys, shares of the key axis, strides, and what lies outside the sequences."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
import attn_ref as ref

pytestmark = pytest.mark.gpu


def run(dev, hq, hk, dim, q_lens, k_lens, causal, seed=0, scale=None, pad=0, std=1.0, gap=0, loose=0):
    """One call on packed sequences (gap: unused rows behind each; loose: how far the maxima lie above the longest);
    o and lse start as NaN."""
    gen = torch.Generator().manual_seed(seed)
    qo, ko = [sum(q_lens[:i]) + gap * i for i in range(len(q_lens) + 1)], [sum(k_lens[:i]) + gap * i for i in range(len(k_lens) + 1)]
    q = ref.bf16(gen, qo[-1], hq * dim, std, pad, dev)
    k = ref.bf16(gen, ko[-1], hk * dim, std, pad, dev)
    v = ref.bf16(gen, ko[-1], hk * dim, 1.0, 2 * pad, dev)
    qs, ks = ref.spans(qo, q_lens), ref.spans(ko, k_lens)
    if gap:      # what lies behind a sequence is never read into a result
        for t, ss, o in ((q, qs, qo), (k, ks, ko), (v, ks, ko)):
            for s, end in zip(ss, o[1:]):
                t[s.stop:end] = float("nan")
    o = torch.full((qo[-1], (hq * dim + 15) // 16 * 16 + pad), float("nan"), dtype=torch.bfloat16, device=dev)[:, :hq * dim]
    lse = torch.full((hq, qo[-1]), float("nan"), device=dev)
    kw = {"q_lengths": ref.i32(q_lens, dev), "k_lengths": ref.i32(k_lens, dev)} if gap else {}
    got = pf.puro_fp8_attention(q, k, v, dim, ref.i32(qo, dev), ref.i32(ko, dev), max(q_lens) + loose,
                                max(k_lens) + loose, causal=causal,
                                scale=scale, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    what = (hq, hk, dim, q_lens, k_lens, causal, scale)
    want, tol, wl, lt = ref.attention(q, k, v, dim, qs, ks, scale or dim ** -0.5, causal)
    ref.close_bf16(o, want, tol, what)
    check_lse(lse, wl, lt, what)


def check_lse(lse, want, tol, what):
    got = ref.f64(lse)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), (what, "rows that see nothing")
    fine = ~inf & ~torch.isnan(want)
    off = (got - want).abs()[fine] - tol[fine]
    assert bool((off <= 0).all()), (what, "lse", float(off.max()))


LENS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", LENS)
def test_one_sequence(dev, n, causal, dim):
    run(dev, 2, 1, dim, [n], [n], causal, seed=n)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (16, 8), (12, 2), (32, 1), (40, 1)])
def test_heads(dev, hq, hk, causal, dim):
    run(dev, hq, hk, dim, [70, 5], [70, 131], causal, seed=hq)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,k", [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 127), (1, 129), (1, 700), (1, 4099), (2, 65),
                                 (7, 300), (16, 1000), (17, 1000), (100, 1300), (300, 3000), (300, 20), (40, 0), (3, 1),
                                 (1, 0), (64, 63), (257, 255)])
def test_other_key_counts(dev, q, k, causal, dim):
    """Single tokens, chunks, and more queries than keys (causal: the first ones see nothing)."""
    run(dev, 4, 2, dim, [q], [k], causal, seed=q + k)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("gap", [0, 3])
def test_packed(dev, causal, dim, gap):
    lens = [5, 0, 130, 1, 64, 257, 0, 33]
    run(dev, 4, 2, dim, lens, lens, causal, seed=1, pad=16, gap=gap)
    run(dev, 4, 2, dim, lens, [9, 4, 130, 0, 90, 300, 0, 32], causal, seed=2, pad=32, gap=gap)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_len", [1, 3])
def test_padded_caches(dev, dim, q_len):
    """Caches whose rows past a sequence's length hold NaN and infinities."""
    hq, hk, cap = 4, 2, 900
    lens = [900, 1, 2, 31, 555, 64, 0]
    gen = torch.Generator().manual_seed(3)
    n = len(lens)
    q = ref.bf16(gen, n * q_len, hq * dim, 1.0, 0, dev)
    k, v = ref.bf16(gen, n * cap, hk * dim, 1.0, 0, dev), ref.bf16(gen, n * cap, hk * dim, 1.0, 0, dev)
    for i, m in enumerate(lens):
        k[i * cap + m:(i + 1) * cap] = float("nan")
        v[i * cap + m:(i + 1) * cap] = float("inf")
    qo, ko = [i * q_len for i in range(n + 1)], [i * cap for i in range(n)]
    o, lse = pf.puro_fp8_attention(q, k, v, dim, ref.i32(qo, dev), ref.i32(ko, dev), q_len, cap,
                                   k_lengths=ref.i32(lens, dev))
    torch.cuda.synchronize()
    want, tol, wl, lt = ref.attention(q, k, v, dim, ref.spans(qo, None), ref.spans(ko, lens), dim ** -0.5, True)
    ref.close_bf16(o, want, tol, "padded")
    check_lse(lse, wl, lt, "padded")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (1e-4, 1.0), (0.125, 6.0), (30.0, 2.0)])
def test_scales(dev, dim, scale, std):
    """Flat rows, and rows whose weight lies on one key."""
    run(dev, 2, 1, dim, [150], [150], True, seed=7, scale=scale, std=std)
    run(dev, 2, 1, dim, [1], [2500], True, seed=8, scale=scale, std=std)


def rising(dev, dim, q_len, k_len):
    """Scores that rise along the keys, so that the running maximum moves at every tile."""
    gen = torch.Generator().manual_seed(11)
    q = ref.bf16(gen, q_len, 2 * dim, 0.1, 0, dev)
    q[:, ::dim] = 4.0
    k, v = ref.bf16(gen, k_len, dim, 0.1, 0, dev), ref.bf16(gen, k_len, dim, 1.0, 0, dev)
    k[:, 0] = torch.linspace(-40.0, 40.0, k_len).to(torch.bfloat16).to(dev)
    return q, k, v


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_len,k_len,down", [(200, 200, False), (200, 200, True), (1, 5000, False), (1, 5000, True),
                                              (300, 2600, False)])
def test_running_maximum(dev, dim, q_len, k_len, down):
    q, k, v = rising(dev, dim, q_len, k_len)
    if down:
        k = k.flip(0).contiguous()
    o, lse = pf.puro_fp8_attention(q, k, v, dim, ref.i32([0, q_len], dev), ref.i32([0, k_len], dev), q_len, k_len,
                                   scale=1.0)
    torch.cuda.synchronize()
    want, tol, wl, lt = ref.attention(q, k, v, dim, [slice(0, q_len)], [slice(0, k_len)], 1.0, True)
    ref.close_bf16(o, want, tol, "rising")
    check_lse(lse, wl, lt, "rising")


def test_maxima_limit_what_is_read(dev):
    """Rows past max_q and max_k, or past the tensor, are left out; wild arrays read and write nothing."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (ref.bf16(gen, 100, 128, 1.0, 0, dev) for _ in range(3))
    o = torch.full((100, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    pf.puro_fp8_attention(q, k, v, 64, ref.i32([0, 100], dev), ref.i32([0, 100], dev), 40, 50, causal=False, o=o)
    torch.cuda.synchronize()
    want, tol, _, _ = ref.attention(q[:40], k[:50], v[:50], 64, [slice(0, 40)], [slice(0, 50)], 0.125, False)
    ref.close_bf16(o[:40], want, tol, "cut")
    assert bool(torch.isnan(o[40:]).all())
    for qo, ko in (([-50, 2 ** 30], [0, 100]), ([2 ** 31 - 1, -2 ** 31], [0, 100]), ([0, 100], [-2 ** 31, 2 ** 31 - 1]),
                   ([0, 100], [99, 2 ** 31 - 1]), ([100, 100], [5, 3])):
        for mq in (100, 1):
            pf.puro_fp8_attention(q, k, v, 64, ref.i32(qo, dev), ref.i32(ko, dev), mq, 100)
    torch.cuda.synchronize()


def test_shared_keys_and_a_longer_output(dev):
    """Two sequences over the same keys; key and value heads as columns of one tensor."""
    gen = torch.Generator().manual_seed(6)
    joint = ref.bf16(gen, 90, 4 * 64, 1.0, 0, dev)
    q, k, v = joint[:, :128], joint[:, 128:192], joint[:, 192:]
    o, _ = pf.puro_fp8_attention(q, k, v, 64, ref.i32([0, 50, 90], dev), ref.i32([0, 0], dev), 50, 90,
                                 k_lengths=ref.i32([90, 90], dev))
    torch.cuda.synchronize()
    want, tol, _, _ = ref.attention(q, k, v, 64, [slice(0, 50), slice(50, 90)], [slice(0, 90)] * 2, 0.125, True)
    ref.close_bf16(o, want, tol, "shared")


def test_equal_calls_give_equal_bits(dev):
    gen = torch.Generator().manual_seed(9)
    for n, m in ((1, 9000), (400, 3000)):
        q, k, v = ref.bf16(gen, n, 4 * 128, 1.0, 0, dev), ref.bf16(gen, m, 2 * 128, 1.0, 0, dev), ref.bf16(gen, m, 2 * 128, 1.0, 0, dev)
        args = (q, k, v, 128, ref.i32([0, n], dev), ref.i32([0, m], dev), n, m)
        a, la = pf.puro_fp8_attention(*args)
        for _ in range(3):
            b, lb = pf.puro_fp8_attention(*args, workspace=torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device=dev))
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_nothing_to_do(dev):
    q, k = torch.empty((0, 128), dtype=torch.bfloat16, device=dev), torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    o, lse = pf.puro_fp8_attention(q, k, k, 64, ref.i32([0], dev), ref.i32([0], dev), 0, 0)
    assert o.shape == (0, 128) and lse.shape == (2, 0)
    gen = torch.Generator().manual_seed(1)
    q = ref.bf16(gen, 5, 128, 1.0, 0, dev)
    o, lse = pf.puro_fp8_attention(q, k, k, 64, ref.i32([0, 5], dev), ref.i32([0, 0], dev), 5, 0)
    torch.cuda.synchronize()
    assert not o.any() and bool((lse == -torch.inf).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,m", [(300, 300), (4, 40), (1, 3000), (2, 9000), (40, 9000)])
def test_a_row_of_nan_is_its_own(dev, n, m, dim):
    """NaN in one query row: its o and lse are NaN, the other rows' are what they are without it."""
    gen = torch.Generator().manual_seed(n + m)
    q, k = ref.bf16(gen, n, 4 * dim, 1.0, 0, dev), ref.bf16(gen, m, 2 * dim, 1.0, 0, dev)
    v = ref.bf16(gen, m, 2 * dim, 1.0, 0, dev)
    plan = (dim, ref.i32([0, n], dev), ref.i32([0, m], dev), n, m)
    o0, l0 = pf.puro_fp8_attention(q, k, v, *plan)
    bad = n // 2
    q[bad, 5] = float("nan")      # of the first head
    o1, l1 = pf.puro_fp8_attention(q, k, v, *plan)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o1[bad, :dim]).all()) and bool(torch.isnan(l1[0, bad]))
    o1[bad, :dim], l1[0, bad] = o0[bad, :dim], l0[0, bad]
    # the maximum is looked for again in the tiles of a wave with a NaN: P may round differently, twice B of sum P |v|
    assert bool(torch.isfinite(o1).all()) and bool(torch.isfinite(l1).all())
    assert float((o1.float() - o0.float()).abs().max()) <= 4 * ref.B * float(v.float().abs().max())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("times", [2, 3, 6])
def test_many_packed_rows(dev, times, causal, dim):
    """About 240, 360 and 720 workgroups of 128 rows: every form of the forward's workgroups."""
    lens = [300, 299, 257, 300, 129] * times
    run(dev, 8, 8, dim, lens, lens, causal, seed=times, gap=2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,k", [(1700, 1700), (200, 2049), (130, 4097), (2100, 2100)])
def test_long_rows(dev, q, k, dim):
    """Both sides of 2048 keys, from which on the keys are split over workgroups."""
    run(dev, 2, 1, dim, [q], [k], True, seed=q)
