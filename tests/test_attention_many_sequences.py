"""The number of sequences that the header promises, where a key head has many query heads: sequences x heads_kv x
ceil(n / 64) below 2^23, n the larger of max_k and max_q heads_q / heads_kv, for both directions."""
import pytest

import test_attention_host as host
import blockwise_fp8_gemm_amd as pf

# heads_q, heads_kv, max_q, max_k
SHAPES = [(64, 1, 1, 1), (64, 1, 1, 64), (1024, 1, 1, 1), (1024, 1, 1, 1024), (1024, 2, 1, 1), (1000, 8, 1, 3), (256, 1, 2, 5),
          (65, 1, 1, 1), (1023, 1, 3, 70), (1024, 512, 1, 1), (1024, 1024, 1, 1), (512, 1, 33, 1), (4, 1, 16, 64)]


def most(hq, hk, q, k):
    """The largest number of sequences within the bound."""
    n = max(k, q * hq // hk)
    return (2 ** 23 - 1) // (hk * -(-n // 64))


def sizes(shape):
    L = pf.lib()
    return L.puro_fp8_attention_workspace_size(shape), L.puro_fp8_attention_bwd_workspace_size(shape)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [2 ** 23, 4096])
@pytest.mark.parametrize("hq,hk,q,k", SHAPES)
def test_promised(hq, hk, q, k, tokens, dim):
    ld = hq * dim if hq * dim % 16 == 0 else 2 ** 22
    for n in (most(hq, hk, q, k), most(hq, hk, q, k) // 2, 1):
        shape = host.attn(heads_q=hq, heads_kv=hk, head_dim=dim, sequences=n, tokens_q=tokens, tokens_k=tokens, max_q=q, max_k=k)
        assert sizes(shape)[1] > 0, n
        # one that fits is told from one that does not by the check that comes next
        lds = dict(ldq=ld, ldk=ld, ldv=ld, ldo=ld)
        assert host._fwd(shape, lse=host.TWO, **lds) == host.ALIGN, n
        assert host._bwd(shape, lse=host.TWO, lddo=ld, lddq=ld, lddk=ld, lddv=ld, **lds) == host.ALIGN, n


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hk,q,k", SHAPES)
def test_more_than_a_grid_has(hq, hk, q, k, dim):
    """Eight times as many sequences pass 2^32 threads in one of the launches of either direction."""
    shape = host.attn(heads_q=hq, heads_kv=hk, head_dim=dim, sequences=min(8 * (most(hq, hk, q, k) + 1), 2 ** 31 - 1),
                      tokens_q=2 ** 23, tokens_k=2 ** 23, max_q=q, max_k=k)
    assert sizes(shape)[1] == 0 and host._bwd(shape) == host.SHAPE
