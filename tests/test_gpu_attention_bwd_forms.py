"""Every form of the gradient's workgroups with several query heads on a key head.  The keys' gradients take one wave of
keys eight times (heads of 64, at most 128 workgroups of 128 keys), two waves four times (fewer than 512) or four waves
twice; the queries' gradients 128 rows on two waves each, or 256."""
import pytest

import test_gpu_attention_bwd as bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk", [(16, 8), (24, 8)])
@pytest.mark.parametrize("times", [1, 3, 6])
def test_packed_grouped_heads(dev, times, hq, hk, causal, dim):
    """120, 360 and 720 workgroups of 128 keys."""
    lens = [300, 299, 257, 300, 129] * times
    bwd.run(dev, hq, hk, dim, lens, lens, causal, seed=times + hq, gap=2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hk,keys", [(16, 1024), (43, 300), (73, 896), (64, 1000)])
def test_where_the_form_changes(dev, hk, keys, causal, dim):
    """128 and 129, 511 and 512 workgroups of 128 keys; each walks the queries of two heads."""
    bwd.run(dev, 2 * hk, hk, dim, [70], [keys], causal, seed=hk)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk", [(5, 1), (12, 4), (7, 7)])
@pytest.mark.parametrize("q,k", [(1, 33), (31, 31), (255, 257), (257, 255), (513, 31), (600, 65)])
def test_narrow_heads_few_keys(dev, q, k, hq, hk, causal):
    """One wave of keys, eight times: fewer queries than its 256 a tile, one more, and several tiles of several heads."""
    bwd.run(dev, hq, hk, 64, [q, 40], [k, 90], causal, seed=q + k + hq)
