"""Timing cases of the attention block between the joint q/k/v product and the output projection.

Each case is one call a training or serving program makes there:

* rope:     norm of every query and key head and the position rotation, in one pass;
* rope_bwd: its gradient, quantised both ways with the values' gradient beside it as the
            joint q/k/v product's dY, and the norm weights' gradients;
* attn:     attention of packed sequences (prompts, chunks of new tokens or single tokens
            over longer key sequences, packed or in padded caches), with the rows' log-sums;
* attn_bwd: the gradients of queries, keys and values.

run() computes the operator in elementary torch operations, or, with `own`,
through the package's entry points.  Codes come back as float8_e4m3fn values
beside their scales.
"""
import torch

own = False

EPS = 1e-6
BASE = 1e6          # base of the rotation's frequencies


def listed():
    def rope(name, op, tokens, hq, hk, dim, rotary, interleaved, norm, start, mscale=1.0, pow2=False):
        return {"name": name, "op": op, "tokens": tokens, "hq": hq, "hk": hk, "dim": dim, "rotary": rotary,
                "interleaved": interleaved, "norm": norm, "start": start, "mscale": mscale, "pow2": pow2}

    def attn(name, op, hq, hk, dim, q_lens, k_lens, causal, capacity=0):
        return {"name": name, "op": op, "hq": hq, "hk": hk, "dim": dim, "q_lens": q_lens, "k_lens": k_lens,
                "causal": causal, "capacity": capacity}

    ragged = "17,1,260,1003,64,2,511,129,1500,33,700"
    return [
        # one token of each of 8 sequences being decoded, far into their contexts: latency only
        rope("rope_8", "rope", 8, 16, 8, 128, 128, False, True, 30000),
        # a prompt chunk of odd length without norms, part of the head rotated, positions of a scaled context
        rope("rope_1037", "rope", 1037, 12, 4, 64, 32, True, False, 900000, 1.2),
        # the training micro-batch (2 x 4096 tokens, 16 / 8 heads of 128)
        rope("rope_8192", "rope", 8192, 16, 8, 128, 128, False, True, 0),
        # the micro-batch's backward
        rope("rope_bwd_8192", "rope_bwd", 8192, 16, 8, 128, 128, False, True, 0),
        # a short odd batch of narrow heads, interleaved pairs, power-of-two scales
        rope("rope_bwd_701", "rope_bwd", 701, 10, 3, 64, 64, True, True, 100, 1.0, True),
        # one new token over one short context: latency only
        attn("attn_decode_1x200", "attn", 16, 8, 128, "1", "200", True),
        # a decoding batch: one new token each over padded caches of 16384 rows
        attn("attn_decode_16", "attn", 16, 8, 128, ",".join(["1"] * 16),
             "16384,517,9000,1,12000,3333,16000,8192,64,15000,7001,2048,11111,5000,16383,129", True, 16384),
        # a chunk of new tokens of one long prompt
        attn("attn_chunk_777x20000", "attn", 16, 8, 128, "777", "20000", True),
        # packed prompts of different lengths, narrow heads
        attn("attn_ragged", "attn", 12, 4, 64, ragged, ragged, True),
        # the training micro-batch
        attn("attn_2x4096", "attn", 16, 8, 128, "4096,4096", "4096,4096", True),
        # its backward
        attn("attn_bwd_2x4096", "attn_bwd", 16, 8, 128, "4096,4096", "4096,4096", True),
        # packed sequences that see all of themselves, narrow heads, backward
        attn("attn_bwd_ragged", "attn_bwd", 12, 4, 64, ragged, ragged, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


HEADS = [(16, 8), (4, 4), (12, 4), (10, 2), (16, 2), (5, 1), (7, 7)]


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "attn", "attn", "attn_bwd"])
    hq, hk = rng.choice(HEADS)
    dim = rng.choice([64, 128])
    if op.startswith("rope"):
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hq, "hk": hk, "dim": dim,
                "rotary": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.7, "start": _log(rng, 1, 1000000), "mscale": rng.choice([1.0, 1.0, 1.3]),
                "pow2": rng.random() < 0.3}
    causal, capacity = rng.random() < 0.7, 0
    if op == "attn" and rng.random() < 0.4:      # a decoding batch, packed keys or padded caches
        n = _log(rng, 1, 24)
        k = [_log(rng, 1, 16384) for _ in range(n)]
        q = [min(v, rng.choice([1, 1, 1, 2, 5])) for v in k]
        capacity = max(k) + rng.randint(0, 100) if rng.random() < 0.5 else 0
    elif op == "attn" and rng.random() < 0.3:    # a chunk of new tokens
        q = [_log(rng, 16, 1500)]
        k = [q[0] + _log(rng, 1, 16384)]
    else:                                        # packed sequences
        n = _log(rng, 1, 12)
        q = [_log(rng, 1, 4096 if n < 4 else 1500) for _ in range(n)]
        k = list(q)
    while sum(a * b for a, b in zip(q, k)) * hq * dim * (1 if causal else 2) > 2 * 4096 * 4096 * 16 * 128:
        q, k = q[:-1], k[:-1]
    if not q:
        q, k, capacity = [300], [300], 0
    return {"op": op, "hq": hq, "hk": hk, "dim": dim, "q_lens": ",".join(map(str, q)),
            "k_lens": ",".join(map(str, k)), "causal": causal, "capacity": capacity}


def _lens(case):
    return [int(v) for v in case["q_lens"].split(",")], [int(v) for v in case["k_lens"].split(",")]


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(rows, cols, std):
        return (torch.randn((rows, cols), generator=gen, device="cuda") * std).to(torch.bfloat16)

    st = dict(case)
    hq, hk, dim = case["hq"], case["hk"], case["dim"]
    if case["op"].startswith("rope"):
        t, half = case["tokens"], case["rotary"] // 2
        # the joint q/k/v product; head outputs of unequal strength
        x = normal(t, (hq + 2 * hk) * dim, 1.0) * torch.linspace(0.5, 2.0, hq + 2 * hk, device="cuda").to(
            torch.bfloat16).repeat_interleave(dim)
        st["q"], st["k"] = x[:, :hq * dim], x[:, hq * dim:(hq + hk) * dim]
        st["positions"] = ((torch.arange(t, device="cuda") * 7) % 4096 + case["start"]).to(torch.int32)
        st["inv_freq"] = (BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        st["wq"] = st["wk"] = None
        if case["norm"]:
            st["wq"], st["wk"] = (1.0 + 0.1 * torch.randn((dim,), generator=gen, device="cuda") for _ in range(2))
        if case["op"] == "rope":
            if t < 64:      # a decoding loop keeps its outputs
                st["q_out"], st["k_out"] = (torch.empty((t, h * dim), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
            return st
        st["rstd"] = None
        if case["norm"]:    # kept by the forward
            st["rstd"] = torch.rsqrt(x[:, :(hq + hk) * dim].double().view(t, hq + hk, dim).square().mean(2) + EPS).float()
        st["dq"], st["dk"], st["dv"] = normal(t, hq * dim, 1e-3), normal(t, hk * dim, 1e-3), normal(t, hk * dim, 1e-3)
        return st
    q_lens, k_lens = _lens(case)
    cap = case["capacity"]
    qo, ko = _offsets(q_lens), [i * cap for i in range(len(k_lens) + 1)] if cap else _offsets(k_lens)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st["q"] = normal(qo[-1], hq * dim, 1.0)
    if cap:     # rows of a cache behind its length hold what was there before
        st["k"], st["v"] = normal(ko[-1], hk * dim, 1.0), normal(ko[-1], hk * dim, 1.0)
        st["k_lengths"] = i32(k_lens)
    else:       # values as the joint product holds them, beside other columns
        st["k"] = normal(ko[-1], hk * dim, 1.0)
        st["v"] = normal(ko[-1], (hq + 2 * hk) * dim, 1.0)[:, (hq + hk) * dim:]
        st["k_lengths"] = None
    st["q_offsets"], st["k_offsets"] = i32(qo), i32(ko)
    st["max_q"], st["max_k"] = max(q_lens), cap or max(k_lens)
    # the rows' sequences and places in them, which the program has beside its offsets
    rep = lambda lens: torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()  # noqa: E731
    place = lambda lens: torch.cat([torch.arange(n) for n in lens]).cuda()  # noqa: E731
    st["q_seq"], st["q_at"] = rep(q_lens), place(q_lens)
    st["k_seq"], st["k_at"] = rep(k_lens), place(k_lens)
    st["q_n"], st["k_n"] = torch.tensor(q_lens).cuda(), torch.tensor(k_lens).cuda()
    if case["op"] == "attn_bwd":
        o, lse, _, _ = _plain_attention(st)     # kept by the forward
        st["o"], st["lse"] = o, lse
        st["do"] = normal(qo[-1], hq * dim, 1e-3)
    return st


def _own(st):
    import blockwise_fp8_gemm_amd as pf
    f8 = torch.float8_e4m3fn
    if st["op"] == "rope":
        q, k, rstd = pf.puro_fp8_qk_norm_rope(
            st["q"], st["k"], st["dim"], st["positions"], st["inv_freq"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
            rope_scale=st["mscale"], interleaved=st["interleaved"], q_out=st.get("q_out"), k_out=st.get("k_out"))
        return {"q": q, "k": k, "rstd": rstd}
    if st["op"] == "rope_bwd":
        _, dwq, dwk, qr, sr, qt, stk = pf.puro_fp8_qk_norm_rope_bwd_quant_dual(
            st["dq"], st["dk"], st["dv"], st["q"], st["k"], st["dim"], st["positions"], st["inv_freq"], rstd=st["rstd"],
            q_weight=st["wq"], k_weight=st["wk"], rope_scale=st["mscale"], interleaved=st["interleaved"], pow2=st["pow2"])
        return {"dwq": dwq, "dwk": dwk, "q_row": qr.view(f8), "s_row": sr, "q_tok": qt.view(f8), "s_tok": stk}
    plan = (st["dim"], st["q_offsets"], st["k_offsets"], st["max_q"], st["max_k"])
    if st["op"] == "attn":
        o, lse = pf.puro_fp8_attention(st["q"], st["k"], st["v"], *plan, k_lengths=st["k_lengths"], causal=st["causal"])
        return {"o": o, "lse": lse}
    dq, dk, dv = pf.puro_fp8_attention_bwd(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], *plan,
                                           k_lengths=st["k_lengths"], causal=st["causal"])
    return {"dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ plain forms

def _plain_scale(amax, pow2):
    if not pow2:
        return amax / 448.0
    m, e = torch.frexp(amax)        # amax = m 2^e, 448 = 0.875 2^9
    k = torch.where(m > 0.875, e - 8, e - 9)
    k = torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(-127, 127)
    return torch.exp2(k.float())


def _plain_rows(n, pow2):
    """1x128 blocks along each row of n [T][C] (FP32)."""
    t, c = n.shape
    nb = (c + 127) // 128
    p = torch.nn.functional.pad(n, (0, nb * 128 - c)).view(t, nb, 128)
    s = _plain_scale(p.abs().amax(2), pow2)
    d = s[:, :, None]
    q = torch.where(d > 0, p / d, p * 0.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(t, nb * 128)[:, :c], s


def _angles(st):
    """cos and sin [tokens][1][rotary / 2] of the rotation, times its scale."""
    a = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    return torch.cos(a).float() * st["mscale"], torch.sin(a).float() * st["mscale"]


def _pairs(x, st):
    """The two members of the rotated pairs of x [T][heads][dim], and the rest of the head."""
    r = st["rotary"]
    if st["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _unpair(a, b, rest, st):
    if st["interleaved"]:
        return torch.cat((torch.stack((a, b), 3).flatten(2), rest), 2)
    return torch.cat((a, b, rest), 2)


def _plain_rope(st, x, w):
    t = x.shape[0]
    x = x.float().view(t, -1, st["dim"])
    rstd = None
    if w is not None:
        rstd = 1.0 / (x.square().mean(2) + EPS).sqrt()
        x = x * rstd[..., None] * w
    cos, sin = _angles(st)
    a, b, rest = _pairs(x, st)
    y = _unpair(a * cos - b * sin, b * cos + a * sin, rest, st)
    return y.reshape(t, -1).to(torch.bfloat16), rstd


def _plain_rope_bwd(st, dy, x, w, rstd):
    t = x.shape[0]
    dy, x = dy.float().view(t, -1, st["dim"]), x.float().view(t, -1, st["dim"])
    cos, sin = _angles(st)
    a, b, rest = _pairs(dy, st)
    g = _unpair(a * cos + b * sin, b * cos - a * sin, rest, st)
    if w is None:
        return g.reshape(t, -1), None
    r = rstd[..., None]
    xh = x * r
    wg = g * w
    dx = r * (wg - xh * (wg * xh).mean(2, keepdim=True))
    return dx.reshape(t, -1), (g * xh).sum((0, 1))


def _padded(x, n, offsets, longest, heads, dim):
    """x's sequences as [sequence][head][longest][dim] in FP32; rows past a length are zero."""
    at = torch.arange(longest, device=x.device)
    rows = (offsets[:-1, None].long() + at).clamp(max=x.shape[0] - 1)
    p = x.view(x.shape[0], heads, dim)[rows] if x.is_contiguous() else x[rows].view(*rows.shape, heads, dim)
    p = torch.where((at < n[:, None])[:, :, None, None], p.float(), 0.0)
    return p.transpose(1, 2).contiguous()


def _plain_attention(st):
    hq, hk, dim, s = st["hq"], st["hk"], st["dim"], st["q_n"].shape[0]
    g, mq, mk = hq // hk, st["max_q"], st["max_k"]
    q = _padded(st["q"], st["q_n"], st["q_offsets"], mq, hq, dim).view(s, hk, g * mq, dim)
    k = _padded(st["k"], st["k_n"], st["k_offsets"], mk, hk, dim)
    v = _padded(st["v"], st["k_n"], st["k_offsets"], mk, hk, dim)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(dim ** -0.5).view(s, hk, g, mq, mk)
    j = torch.arange(mk, device=q.device)
    seen = j < st["k_n"][:, None, None]
    if st["causal"]:
        last = torch.arange(mq, device=q.device) + (st["k_n"] - st["q_n"])[:, None]
        seen = seen & (j <= last[:, :, None])
    x.masked_fill_(~seen[:, None, None], -torch.inf)
    top = x.amax(4, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(4, keepdim=True)
    lse = (top + torch.log(total)).view(s, hq, mq)
    x = x.div_(torch.where(total > 0, total, 1.0))
    o = torch.matmul(x.view(s, hk, g * mq, mk), v).view(s, hq, mq, dim)
    # back to the packed rows
    o = o[st["q_seq"], :, st["q_at"]].reshape(-1, hq * dim).to(torch.bfloat16)
    return o, lse[st["q_seq"], :, st["q_at"]].t().contiguous(), x, (q, k, v)


def _plain_attention_bwd(st):
    hq, hk, dim, s = st["hq"], st["hk"], st["dim"], st["q_n"].shape[0]
    g, mq, mk = hq // hk, st["max_q"], st["max_k"]
    _, _, p, (q, k, v) = _plain_attention(st)
    p = p.view(s, hk, g * mq, mk)
    do = _padded(st["do"], st["q_n"], st["q_offsets"], mq, hq, dim).view(s, hk, g * mq, dim)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(3, keepdim=True)) * dim ** -0.5
    dq = torch.matmul(ds, k).view(s, hq, mq, dim)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    dq = dq[st["q_seq"], :, st["q_at"]].reshape(-1, hq * dim)
    dk, dv = (t[st["k_seq"], :, st["k_at"]].reshape(-1, hk * dim) for t in (dk, dv))
    return {"dq": dq.to(torch.bfloat16), "dk": dk.to(torch.bfloat16), "dv": dv.to(torch.bfloat16)}


def _plain(st):
    if st["op"] == "rope":
        q, rq = _plain_rope(st, st["q"], st["wq"])
        k, rk = _plain_rope(st, st["k"], st["wk"])
        return {"q": q, "k": k, "rstd": torch.cat((rq, rk), 1) if st["norm"] else None}
    if st["op"] == "rope_bwd":
        rq, rk = (st["rstd"][:, :st["hq"]], st["rstd"][:, st["hq"]:]) if st["norm"] else (None, None)
        dq, dwq = _plain_rope_bwd(st, st["dq"], st["q"], st["wq"], rq)
        dk, dwk = _plain_rope_bwd(st, st["dk"], st["k"], st["wk"], rk)
        dx = torch.cat((dq, dk, st["dv"].float()), 1)
        qr, sr = _plain_rows(dx, st["pow2"])
        qt, stk = _plain_rows(dx.t().contiguous(), st["pow2"])
        return {"dwq": dwq, "dwk": dwk, "q_row": qr, "s_row": sr, "q_tok": qt, "s_tok": stk}
    if st["op"] == "attn":
        o, lse, _, _ = _plain_attention(st)
        return {"o": o, "lse": lse}
    return _plain_attention_bwd(st)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors

def _pairs_seen(case):
    q_lens, k_lens = _lens(case)
    if not case["causal"]:
        return sum(a * b for a, b in zip(q_lens, k_lens))
    # query i of n sees keys 0 .. i + m - n
    return sum(sum(max(0, min(m, i + m - n + 1)) for i in range(n)) for n, m in zip(q_lens, k_lens))


def work(case):
    hq, hk, dim = case["hq"], case["hk"], case["dim"]
    if case["op"].startswith("rope"):
        t, c = case["tokens"], (hq + hk) * dim
        extra = 4 * t + 2 * case["rotary"] + (8 * dim + 4 * t * (hq + hk) if case["norm"] else 0)
        if case["op"] == "rope":
            return {"bytes": 4 * t * c + extra, "flops": 10 * t * c}
        j = (hq + 2 * hk) * dim
        # without norms the products' q and k do not enter
        moved = (4 if case["norm"] else 2) * t * c + 2 * t * hk * dim + 2 * t * j
        scales = 4 * t * ((j + 127) // 128) + 4 * j * ((t + 127) // 128)
        return {"bytes": moved + scales + extra + (8 * dim if case["norm"] else 0), "flops": 20 * t * c}
    q_lens, k_lens = _lens(case)
    tq, tk, pairs = sum(q_lens), sum(k_lens), _pairs_seen(case)
    if case["op"] == "attn":
        return {"bytes": 4 * tq * hq * dim + 4 * tk * hk * dim + 4 * tq * hq, "flops": 4 * dim * hq * pairs}
    return {"bytes": 8 * tq * hq * dim + 8 * tk * hk * dim + 4 * tq * hq, "flops": 10 * dim * hq * pairs}


# ------------------------------------------------------------------ 64-bit results

def _e4m3_64(y):
    """Nearest E4M3 value (ties to even) of float64 values with |y| <= 448."""
    mag = y.abs()
    _, e = torch.frexp(mag)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)     # 3 mantissa bits, subnormals below 2^-6
    return torch.copysign((torch.round(mag / step) * step).clamp(max=448.0), y)


def _exact_blocks(v, dim, pow2):
    """Codes' values and scales of 128-long blocks of v (float64) along dim."""
    codes, scales = [], []
    for p in torch.split(v, 128, dim):
        top = p.abs().amax(dim, keepdim=True)
        s = top / 448.0
        if pow2:
            s = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(s))).clamp(2.0 ** -127, 2.0 ** 127),
                            torch.full_like(top, 2.0 ** -127))
        codes.append(torch.where(s > 0, _e4m3_64(p / s), p * 0.0))
        scales.append(s)
    return torch.cat(codes, dim), torch.cat(scales, dim)


def _exact_rotation(st):
    """The rotation of a head as complex factors [tokens][rotary / 2], and the columns of the pairs."""
    turn = torch.polar(torch.full_like(st["inv_freq"], st["mscale"], dtype=torch.float64).expand(st["tokens"], -1),
                       torch.outer(st["positions"].double(), st["inv_freq"].double()))
    i = torch.arange(st["rotary"] // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + st["rotary"] // 2)
    return turn, first, second


def _exact_turn(v, turn, first, second):
    """v [T][heads][dim] (float64) with its pairs multiplied by turn as complex numbers."""
    z = torch.complex(v[..., first], v[..., second]) * turn[:, None]
    out = v.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(st):
    turn, first, second = _exact_rotation(st)
    outs, rs = [], []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        v = x.double().reshape(st["tokens"], -1, st["dim"])
        if w is not None:
            rms = (torch.linalg.vector_norm(v, dim=2) ** 2 / st["dim"] + EPS).sqrt()
            rs.append(1.0 / rms)
            v = v / rms[..., None] * w.double()
        outs.append(_exact_turn(v, turn, first, second).flatten(1))
    return {"q": outs[0], "k": outs[1], "rstd": torch.cat(rs, 1) if rs else None}


def _exact_rope_bwd(st):
    turn, first, second = _exact_rotation(st)
    hq, parts, out = st["hq"], [], {"dwq": None, "dwk": None}
    for name, dy, x, w, heads in (("dwq", st["dq"], st["q"], st["wq"], slice(0, hq)),
                                  ("dwk", st["dk"], st["k"], st["wk"], slice(hq, None))):
        # the transpose of a rotation times a factor is the conjugate factor
        g = _exact_turn(dy.double().reshape(st["tokens"], -1, st["dim"]), turn.conj(), first, second)
        if w is not None:
            r = st["rstd"][:, heads].double()[..., None]
            v = x.double().reshape(st["tokens"], -1, st["dim"])
            out[name] = torch.einsum("thd,thd->d", g, v * r)
            wg = g * w.double()
            g = wg * r - v * (wg * v).sum(2, keepdim=True) * r ** 3 / st["dim"]
        parts.append(g.flatten(1))
    dx = torch.cat((*parts, st["dv"].double()), 1)
    out["q_row"], out["s_row"] = _exact_blocks(dx, 1, st["pow2"])
    qt, stk = _exact_blocks(dx, 0, st["pow2"])
    return out | {"q_tok": qt.t().contiguous(), "s_tok": stk.t().contiguous()}


def _exact_attention(st, case):
    """A sequence and a query head at a time, in 64 bits."""
    hq, hk, dim = st["hq"], st["hk"], st["dim"]
    q_lens, k_lens = _lens(case)
    qo, ko = st["q_offsets"].tolist(), st["k_offsets"].tolist()
    back = case["op"] == "attn_bwd"
    names = ("dq", "dk", "dv") if back else ("o",)
    res = {"dq": st["q"], "dk": st["k"], "dv": st["k"], "o": st["q"]}
    res = {n: torch.zeros(res[n].shape, dtype=torch.float64, device="cuda") for n in names}
    lse = torch.full((hq, qo[-1]), -torch.inf, dtype=torch.float64, device="cuda")
    for s, (n, m) in enumerate(zip(q_lens, k_lens)):
        rows, keys = slice(qo[s], qo[s] + n), slice(ko[s], ko[s] + m)
        hide = None
        if case["causal"]:
            hide = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(hq):
            qc, kc = slice(h * dim, (h + 1) * dim), slice(h // (hq // hk) * dim, (h // (hq // hk) + 1) * dim)
            q, k, v = st["q"][rows, qc].double(), st["k"][keys, kc].double(), st["v"][keys, kc].double()
            x = q @ k.t().contiguous() / dim ** 0.5
            if hide is not None:
                x = x.masked_fill(hide, -torch.inf)
            lse[h, rows] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1).nan_to_num(0.0)
            if not back:
                res["o"][rows, qc] = p @ v
                continue
            do = st["do"][rows, qc].double()
            o = p @ v
            ds = p * (do @ v.t().contiguous() - (do * o).sum(1, keepdim=True)) / dim ** 0.5
            res["dq"][rows, qc] = ds @ k
            res["dk"][keys, kc] += ds.t().contiguous() @ q
            res["dv"][keys, kc] += p.t().contiguous() @ do
    return res if back else {"o": res["o"], "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "rope_bwd":
        return _exact_rope_bwd(st)
    return _exact_attention(st, case)
