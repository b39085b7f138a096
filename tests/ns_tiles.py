"""Which tile the orthogonalisation's launches take, as launch_product in newton.hip chooses: the form with
the least estimated time.  Tile shapes, grouping limit and times are read from the source."""
import math
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_fp8_gemm_amd", "csrc")
GRAM, POLY, UPDATE = "X X^T", "A A", "B X"


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def forms():
    """[(rows, columns of the tile, fixed, one, many)] of the four forms, largest first."""
    text = _read("newton.hip")
    tiles = {m[5]: (int(m[0]) * int(m[2]) * 16, int(m[1]) * int(m[3]) * 16)
             for m in re.findall(r"typedef NsCfg<(\d+), (\d+), (\d+), (\d+), (\d+)> (Ns\w)", text)}
    times = re.findall(r"estimate<(Ns\w), MODE>\(g, ([\d.]+), ([\d.]+), ([\d.]+)\)", text)
    assert len(tiles) == len(times) == 4, (tiles, times)
    return [tiles[n] + (float(f), float(o), float(m)) for n, f, o, m in times]


def group_max():
    return int(re.search(r"constexpr int kNsGroupMax = (\d+);", _read("kernels.h")).group(1))


def tile(shapes, product):
    """(rows, columns) of the tile that one launch over these matrices takes for a product."""
    assert len(shapes) <= group_max()
    up = [tuple(-(-n // 128) * 128 for n in sorted(s)) for s in shapes]      # (Mp, Np)
    depth = [(n if product == GRAM else m) // 64 for m, n in up]
    order = sorted(range(len(up)), key=lambda i: -depth[i])
    best = None
    for tm, tn, fixed, one, many in forms():
        if any(m % tn or (n if product == UPDATE else m) % tm for m, n in up):
            continue
        count = work = most = 0
        for i in order:
            m, n = up[i]
            rows = (n if product == UPDATE else m) // tm
            tiles = rows * (m // tn) - (0 if product == UPDATE else tm // tn * (rows * (rows - 1) // 2))
            count += tiles
            work += tiles * depth[i]
            most = max(most, math.ceil(count / 256) * depth[i])
        t = fixed + max(most, work / 256) * (one if count <= 256 else many)
        if best is None or t < best[0]:
            best = (t, (tm, tn))
    return best[1]


def tiles(shapes):
    return tuple(tile(shapes, p) for p in (GRAM, POLY, UPDATE))


# Groups that between them take every form for every product; ragged, tall and wide matrices.  The seven
# gradients of a Qwen3-1.7B layer are one of them.
GROUPS = {
    "small": [(200, 520), (520, 200), (129, 64)],
    "one square": [(2048, 2048)],
    "two": [(1500, 2000), (2000, 1500)],
    "mixed": [(1000, 1000)] * 8 + [(250, 1500), (1500, 250)] * 4,
    "eight": [(1000, 1500), (1500, 1000)] * 4,
    "sixteen": [(1000, 1500), (1500, 1000)] * 8,
    "layer": [(2048, 2048), (1024, 2048), (1024, 2048), (2048, 2048), (6144, 2048), (6144, 2048), (2048, 6144)],
}
TILES = {   # of X X^T, A A and B X
    "small": ((64, 64), (64, 64), (64, 64)),
    "one square": ((128, 128), (128, 128), (128, 128)),
    "two": ((128, 128), (128, 128), (256, 128)),
    "mixed": ((128, 128), (256, 128), (256, 128)),
    "eight": ((256, 128), (256, 128), (256, 256)),
    "sixteen": ((256, 256), (256, 256), (256, 256)),
    "layer": ((256, 128), (256, 256), (256, 256)),
}
