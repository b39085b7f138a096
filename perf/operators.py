"""Timing cases of the operators around the blockwise-FP8 GEMMs.

Each case is one call a training or serving program makes between two GEMMs:

* norm:       residual addition, root-mean-square norm and E4M3 block quantisation
              (row blocks only for serving, row and token blocks for training);
* norm_bwd:   the norm's gradient, quantised both ways as the gradient of the
              linear layer before it, and the norm weight's gradient;
* swiglu_bwd: the gated activation's gradient, quantised both ways side by side;
* ns:         weight gradients orthogonalised by Newton-Schulz products.

run() computes the operator in elementary torch operations, or, with `own`,
through the package's entry points.  Codes come back as float8_e4m3fn values
beside their scales.
"""
import torch

own = False

EPS = 1e-6
NS = (3.4445, -4.7750, 2.0315)      # quintic of the orthogonalisation
NS_STEPS = 5
NS_EPS = 1e-7

# rows x cols of one decoder layer's seven weight gradients (q, k, v, o, gate, up, down)
LAYER = "2048x2048,1024x2048,1024x2048,2048x2048,6144x2048,6144x2048,2048x6144"


def listed():
    def norm(name, tokens, cols, dual, residual, w="f32", pow2=False):
        return {"name": name, "op": "norm", "tokens": tokens, "cols": cols, "dual": dual,
                "residual": residual, "w": w, "pow2": pow2}

    def bwd(name, tokens, cols, residual, w="f32", pow2=False):
        return {"name": name, "op": "norm_bwd", "tokens": tokens, "cols": cols, "residual": residual, "w": w,
                "pow2": pow2}

    def swiglu(name, tokens, cols, joined, pow2=False):
        return {"name": name, "op": "swiglu_bwd", "tokens": tokens, "cols": cols, "joined": joined, "pow2": pow2}

    def ns(name, shapes, dtype):
        return {"name": name, "op": "ns", "shapes": shapes, "dtype": dtype}

    return [
        # one token of one sequence being decoded: latency only
        norm("norm_1x2048", 1, 2048, False, True),
        # a prompt chunk of odd length, served (row blocks only), BF16 norm weight
        norm("norm_1037x2048", 1037, 2048, False, True, "bf16"),
        # the training micro-batch in front of q/k/v or gate/up
        norm("norm_8192x2048", 8192, 2048, True, True),
        # no residual, ragged width and tokens, power-of-two scales for the scaled matrix cores
        norm("norm_517x1500", 517, 1500, True, False, "bf16", True),
        # the micro-batch's backward, the residual's gradient joining in
        bwd("norm_bwd_8192x2048", 8192, 2048, True),
        # a short odd batch without a residual branch
        bwd("norm_bwd_700x1100", 700, 1100, False, "bf16"),
        # the feed-forward's backward of the micro-batch, gate and up gradients side by side
        swiglu("swiglu_bwd_8192x6144", 8192, 6144, True),
        # ragged feed-forward width: separate outputs
        swiglu("swiglu_bwd_333x1000", 333, 1000, False),
        # one square projection's update
        ns("ns_2048x2048", "2048x2048", "f32"),
        # all seven updates of a layer in one call
        ns("ns_layer", LAYER, "f32"),
        # small odd matrices, tall and wide, BF16 momentum
        ns("ns_small", "200x520,520x200,129x64", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "swiglu_bwd", "ns"])
    w = rng.choice(["f32", "bf16"])
    if op == "norm":
        dual = rng.random() < 0.5
        return {"op": op, "tokens": _log(rng, 1, 8192), "cols": _log(rng, 64, 6144), "dual": dual,
                "residual": rng.random() < 0.7, "w": w, "pow2": False}
    if op == "norm_bwd":
        return {"op": op, "tokens": _log(rng, 1, 8192), "cols": _log(rng, 64, 6144), "residual": rng.random() < 0.7,
                "w": w, "pow2": False}
    if op == "swiglu_bwd":
        joined = rng.random() < 0.5
        cols = _log(rng, 64, 6144)
        if joined:      # the two gradients' blocks meet at a block boundary
            cols = max(128, cols // 128 * 128)
        return {"op": op, "tokens": _log(rng, 1, 8192), "cols": cols, "joined": joined, "pow2": False}
    shapes = []
    for _ in range(rng.randint(1, 3)):
        a = _log(rng, 32, 2048)
        b = min(6144, _log(rng, a, 4 * a))
        shapes.append("%dx%d" % ((a, b) if rng.random() < 0.5 else (b, a)))
    return {"op": op, "shapes": ",".join(shapes), "dtype": rng.choice(["f32", "bf16"])}


def _pad16(n):
    return (n + 15) // 16 * 16


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(rows, cols, std):
        # rows at a stride of a multiple of 16 elements, as the package's tensors have
        t = torch.randn((rows, _pad16(cols)), generator=gen, device="cuda") * std
        return t.to(torch.bfloat16)[:, :cols]

    st = dict(case)
    if case["op"] == "ns":
        st["grads"] = []
        for r, c in _shapes(case):
            # a gradient's decaying spectrum: a few strong directions over a broad floor
            k = min(16, r, c)
            g = torch.randn((r, k), generator=gen, device="cuda") @ torch.randn((k, c), generator=gen, device="cuda")
            g = 1e-4 * (0.05 * g + torch.randn((r, c), generator=gen, device="cuda"))
            ld = _pad16(c)
            buf = torch.zeros((r, ld), device="cuda", dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
            buf[:, :c] = g
            st["grads"].append(buf[:, :c])
        return st
    t, c = case["tokens"], case["cols"]
    if case["op"] == "swiglu_bwd":
        # the gate/up product (or its two halves' tensors) and the down projection's data gradient
        if case["joined"]:
            gu = normal(t, 2 * c, 1.0)
            st["gate"], st["up"] = gu[:, :c], gu[:, c:]
        else:
            st["gate"], st["up"] = normal(t, c, 1.0), normal(t, c, 1.0)
        st["dh"] = normal(t, c, 1e-3)
        return st
    w = 1.0 + 0.1 * torch.randn((c,), generator=gen, device="cuda")
    st["weight"] = w if case["w"] == "f32" else w.to(torch.bfloat16)
    # residual streams carry a few channels far above the rest
    loud = 1.0 + 30.0 * (torch.rand((c,), generator=gen, device="cuda") < 0.01)
    if case["op"] == "norm":
        st["x"] = normal(t, c, 1.0)
        st["residual"] = (normal(t, c, 2.0) * loud.to(torch.bfloat16)) if case["residual"] else None
        if st["residual"] is not None:
            st["residual"] = _strided(st["residual"])
        if not case["dual"]:
            # a serving loop keeps its output buffers
            nb = (c + 127) // 128
            st["bufs"] = {"q": torch.empty((t, _pad16(c)), dtype=torch.uint8, device="cuda")[:, :c],
                          "s": torch.empty((t, nb), device="cuda"), "rstd": torch.empty((t,), device="cuda")}
            if st["residual"] is not None:
                st["bufs"]["z"] = torch.empty((t, _pad16(c)), dtype=torch.bfloat16, device="cuda")[:, :c]
        return st
    z = _strided(normal(t, c, 2.0) * loud.to(torch.bfloat16))
    st["z"] = z
    st["rstd"] = torch.rsqrt(z.double().square().mean(1) + EPS).float()   # kept by the forward
    st["dy"] = normal(t, c, 1e-3)
    st["dres"] = normal(t, c, 1e-3) if case["residual"] else None
    return st


def _strided(t):
    buf = torch.zeros((t.shape[0], _pad16(t.shape[1])), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _own(st):
    import blockwise_fp8_gemm_amd as pf
    f8 = torch.float8_e4m3fn
    if st["op"] == "norm":
        if st["dual"]:
            z, rstd, _, qr, sr, qt, stk = pf.puro_fp8_rmsnorm_quant_dual(
                st["x"], st["weight"], st["residual"], eps=EPS, pow2=st["pow2"])
            out = {"rstd": rstd, "q_row": qr.view(f8), "s_row": sr, "q_tok": qt.view(f8), "s_tok": stk}
        else:
            z, rstd, _, qr, sr = pf.puro_fp8_rmsnorm_quant_act(
                st["x"], st["weight"], st["residual"], eps=EPS, pow2=st["pow2"], **st["bufs"])
            out = {"rstd": rstd, "q_row": qr.view(f8), "s_row": sr}
        if st["residual"] is not None:
            out["z"] = z
        return out
    if st["op"] == "norm_bwd":
        dx, dw, qr, sr, qt, stk = pf.puro_fp8_rmsnorm_bwd_quant_dual(
            st["dy"], st["z"], st["rstd"], st["weight"], st["dres"], pow2=st["pow2"])
        return {"dx": dx, "dw": dw, "q_row": qr.view(f8), "s_row": sr, "q_tok": qt.view(f8), "s_tok": stk}
    if st["op"] == "swiglu_bwd":
        got = pf.puro_fp8_swiglu_bwd_quant_dual(st["dh"], st["gate"], st["up"], joined=st["joined"], pow2=st["pow2"])
        if st["joined"]:
            qr, sr, qt, stk = got
            return {"q_row": qr.view(f8), "s_row": sr, "q_tok": qt.view(f8), "s_tok": stk}
        return [{"q_row": qr.view(f8), "s_row": sr, "q_tok": qt.view(f8), "s_tok": stk} for qr, sr, qt, stk in got]
    return pf.puro_fp8_newton_schulz_grouped(st["grads"], steps=NS_STEPS, coefficients=NS, eps=NS_EPS)


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


def _plain_dual(n, pow2):
    qr, sr = _plain_rows(n, pow2)
    qt, stk = _plain_rows(n.t().contiguous(), pow2)     # 128-token blocks of each column, transposed
    return {"q_row": qr, "s_row": sr, "q_tok": qt, "s_tok": stk}


def _plain_ns(g):
    x = g.float()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (x.square().sum().sqrt() + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        m = x @ x.t()
        x = a * x + (b * m + c * (m @ m)) @ x
    return (x.t() if tall else x).to(torch.bfloat16)


def _plain(st):
    if st["op"] == "ns":
        return [_plain_ns(g) for g in st["grads"]]
    if st["op"] == "swiglu_bwd":
        dh, g, u = st["dh"].float(), st["gate"].float(), st["up"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        dg = dh * u * sig * (1.0 + g * (1.0 - sig))
        du = dh * g * sig
        if st["joined"]:
            return _plain_dual(torch.cat((dg, du), 1), st["pow2"])
        return [_plain_dual(dg, st["pow2"]), _plain_dual(du, st["pow2"])]
    w = st["weight"].float()
    if st["op"] == "norm":
        z = st["x"]
        if st["residual"] is not None:
            z = (z.float() + st["residual"].float()).to(torch.bfloat16)
        zf = z.float()
        rstd = 1.0 / (zf.square().mean(1) + EPS).sqrt()
        n = zf * rstd[:, None] * w
        if st["dual"]:
            out = _plain_dual(n, st["pow2"])
        else:
            out = dict(zip(("q_row", "s_row"), _plain_rows(n, st["pow2"])))
        out["rstd"] = rstd
        if st["residual"] is not None:
            out["z"] = z
        return out
    dy, xh, r = st["dy"].float(), st["z"].float() * st["rstd"][:, None], st["rstd"][:, None]
    g = dy * w
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    out = _plain_dual(dx, st["pow2"])
    out["dx"] = dx.to(torch.bfloat16)
    out["dw"] = (dy * xh).sum(0)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors

def work(case):
    if case["op"] == "ns":
        flops = bytes_ = 0
        for r, c in _shapes(case):
            m, n = min(r, c), max(r, c)
            # X X^T and A A are symmetric: half of each; B X in full
            flops += NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)
            bytes_ += r * c * ((4 if case["dtype"] == "f32" else 2) + 2)
        return {"bytes": bytes_, "flops": flops}
    t, c = case["tokens"], case["cols"]
    row, tok = t * c + 4 * t * ((c + 127) // 128), t * c + 4 * c * ((t + 127) // 128)
    if case["op"] == "swiglu_bwd":
        return {"bytes": 6 * t * c + 2 * (row + tok), "flops": 20 * t * c}
    wb = c * (4 if case["w"] == "f32" else 2)
    if case["op"] == "norm":
        moved = t * c * (6 if case["residual"] else 2) + wb + 4 * t
        return {"bytes": moved + row + (tok if case["dual"] else 0), "flops": 8 * t * c}
    moved = t * c * (8 if case["residual"] else 6) + wb + 4 * t + 4 * c
    return {"bytes": moved + row + tok, "flops": 14 * t * c}


# ------------------------------------------------------------------ 64-bit results

def _e4m3_64(y):
    """Nearest E4M3 value (ties to even) of float64 values with |y| <= 448."""
    mag = y.abs()
    _, e = torch.frexp(mag)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)     # 3 mantissa bits, subnormals below 2^-6
    return torch.copysign((torch.round(mag / step) * step).clamp(max=448.0), y)


def _exact_blocks(v, dim, pow2):
    """Codes' values and scales of 128-long blocks of v (float64) along dim."""
    parts = torch.split(v, 128, dim)
    codes, scales = [], []
    for p in parts:
        top = p.abs().amax(dim, keepdim=True)
        s = top / 448.0
        if pow2:
            s = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(s))).clamp(2.0 ** -127, 2.0 ** 127),
                            torch.full_like(top, 2.0 ** -127))
        codes.append(torch.where(s > 0, _e4m3_64(p / s), p * 0.0))
        scales.append(s)
    return torch.cat(codes, dim), torch.cat(scales, dim)


def _exact_dual(v, pow2):
    qr, sr = _exact_blocks(v, 1, pow2)
    qt, stk = _exact_blocks(v, 0, pow2)
    return {"q_row": qr, "s_row": sr, "q_tok": qt.t().contiguous(), "s_tok": stk.t().contiguous()}


def _exact_ns(g):
    # the steps commute with X X^T: O = H X with H a polynomial of the Gram matrix
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    x = x / (torch.linalg.vector_norm(x) + NS_EPS)
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    gram, h = x @ x.t().contiguous(), eye
    a, b, c = NS
    for _ in range(NS_STEPS):
        f = a * eye + gram @ (b * eye + c * gram)
        h = h @ f
        gram = f @ gram @ f
    x = h @ x
    return x.t() if tall else x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ns":
        return [_exact_ns(g) for g in st["grads"]]
    if case["op"] == "swiglu_bwd":
        dh, g, u = st["dh"].double(), st["gate"].double(), st["up"].double()
        sig = torch.sigmoid(g)
        grads = (dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * g * sig)
        if case["joined"]:
            return _exact_dual(torch.cat(grads, 1), case["pow2"])
        return [_exact_dual(v, case["pow2"]) for v in grads]
    w = st["weight"].double()
    if case["op"] == "norm":
        z = st["x"].double()
        out = {}
        if st["residual"] is not None:
            # the residual stream is a BF16 tensor: the norm is of what it holds
            z = st["x"].float().add(st["residual"].float()).bfloat16().double()
            out["z"] = z
        rms = (torch.einsum("tc,tc->t", z, z) / z.shape[1] + EPS).sqrt()
        v = z / rms[:, None] * w
        if case["dual"]:
            out |= _exact_dual(v, case["pow2"])
        else:
            out["q_row"], out["s_row"] = _exact_blocks(v, 1, case["pow2"])
        out["rstd"] = 1.0 / rms
        return out
    dy, z, r = st["dy"].double(), st["z"].double(), st["rstd"].double()
    inner = (dy * w * z).sum(1) * r ** 3 / z.shape[1]
    dx = dy * w * r[:, None] - z * inner[:, None]
    if st["dres"] is not None:
        dx = dx + st["dres"].double()
    out = _exact_dual(dx, case["pow2"])
    out["dx"] = dx
    out["dw"] = (dy * z * r[:, None]).sum(0)
    return out
