"""The groups of matrices that the GPU tests orthogonalise take every tile form of every product."""
import pytest

from ns_tiles import GROUPS, TILES, forms, tiles


@pytest.mark.parametrize("name", sorted(GROUPS))
def test_group_takes_its_tiles(name):
    assert tiles(GROUPS[name]) == TILES[name]


def test_every_form_of_every_product():
    shapes = {f[:2] for f in forms()}
    assert shapes == {(256, 256), (256, 128), (128, 128), (64, 64)}
    for product in range(3):
        assert {t[product] for t in TILES.values()} == shapes


def test_measured_choices():
    """The choices that the comment at launch_product gives the measured times of."""
    n = 2048
    assert tiles([(1024, 1024)])[0] == (64, 64) and tiles([(1024, 4096)])[0] == (64, 64)
    assert tiles([(n, n)])[0] == (128, 128) and tiles([(n, n)] * 2)[0] == (256, 128)
    assert tiles([(n, n)])[2] == (128, 128) and tiles([(n, n)] * 2)[2] == (256, 128)
