"""The activation gradient's separate results written into tensors that the caller keeps."""
import pytest
import torch

import blockwise_fp8_gemm_amd as pf
from fused_ref import bf16

pytestmark = pytest.mark.gpu


def kept(tokens, cols, transpose_out, dev):
    """Pairs of every output, in rows wider than they need, filled with a mark."""
    tok = (cols, tokens) if transpose_out else (tokens, cols)
    nt = -(-tokens // 128)

    def codes(rows, n):
        return torch.full((rows, (n + 15) // 16 * 16 + 32), 0x5A, dtype=torch.uint8, device=dev)

    def scales(*shape):
        return torch.full(shape, -7.0, device=dev)
    return {"q_row": [codes(tokens, cols) for _ in range(2)], "q_tok": [codes(*tok) for _ in range(2)],
            "s_row": [scales(tokens, -(-cols // 128)) for _ in range(2)],
            "s_tok": [scales(*((cols, nt) if transpose_out else (nt, cols))) for _ in range(2)]}, tok[1]


@pytest.mark.parametrize("pow2", [False, True], ids=["amax", "pow2"])
@pytest.mark.parametrize("transpose_out", [True, False], ids=["nt", "tn"])
@pytest.mark.parametrize("tokens,cols", [(1, 1), (1, 300), (333, 1000), (130, 129), (128, 256)])
def test_given_outputs(dev, tokens, cols, transpose_out, pow2):
    dh, gate, up = (bf16(tokens, cols, 1.0, k, dev, 16) for k in (1, 2, 3))
    want = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, transpose_out=transpose_out, pow2=pow2)
    bufs, width = kept(tokens, cols, transpose_out, dev)
    outs = {"q_row": [b[:, :cols] for b in bufs["q_row"]], "q_tok": tuple(b[:, :width] for b in bufs["q_tok"]),
            "s_row": bufs["s_row"], "s_tok": bufs["s_tok"]}
    for _ in range(2):
        got = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, transpose_out=transpose_out, pow2=pow2, **outs)
    torch.cuda.synchronize()
    for k in range(2):
        for w, g, name in zip(want[k], got[k], ("q_row", "s_row", "q_tok", "s_tok")):
            assert torch.equal(w, g) and g.data_ptr() == outs[name][k].data_ptr(), (k, name)
        assert bool((bufs["q_row"][k][:, cols:] == 0x5A).all()) and bool((bufs["q_tok"][k][:, width:] == 0x5A).all())
    # some given, the others allocated
    part = pf.puro_fp8_swiglu_bwd_quant_dual(dh, gate, up, transpose_out=transpose_out, pow2=pow2,
                                             q_tok=(None, outs["q_tok"][1]), s_row=(outs["s_row"][0], None))
    torch.cuda.synchronize()
    assert part[1][2].data_ptr() == outs["q_tok"][1].data_ptr() and part[0][1].data_ptr() == outs["s_row"][0].data_ptr()
    assert all(torch.equal(w, g) for k in range(2) for w, g in zip(want[k], part[k]))


def test_refusals(dev):
    x = bf16(40, 200, 1.0, 1, dev)
    q = torch.empty((40, 208), dtype=torch.uint8, device=dev)[:, :200]
    for bad in (q, (q,), (q, q, q)):
        with pytest.raises(ValueError, match="pair"):
            pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x, q_row=bad)
    with pytest.raises(ValueError, match="expected"):
        pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x, q_row=(None, q[:, :100]))
    with pytest.raises(ValueError, match="expected"):
        pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x, s_tok=(torch.empty((200, 2), device=dev), None))
    with pytest.raises(ValueError, match="GPU"):
        pf.puro_fp8_swiglu_bwd_quant_dual(x, x, x, q_row=(q.cpu(), q))
