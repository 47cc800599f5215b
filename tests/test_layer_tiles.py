"""The cases of the tile tests still reach the shapes and the tiles a workgroup that they name."""
import re

import numpy as np
import pytest

import layer_tiles as tiles
from test_gpu_layer import counts_of


def counts(T, E, N, K, kind):
    return counts_of(kind, E, T, np.random.default_rng(T + N + K))


def test_the_rule_is_the_source_s():
    """The numbers that the rule repeats stand in the source as they do here."""
    text = open(tiles.SOURCE).read()
    for name, value in (("kStepK", tiles.KSTEP), ("kXcds", tiles.XCDS), ("kCus", tiles.CUS),
                        ("kRing", tiles.RING)):
        assert re.search(rf"constexpr int {name} = {value};", text), name
    shapes = [(int(m), int(n), g) for m, n, g in
              re.findall(r"launch_tile<(\d+), (\d+), \d+, \d+, \d+, \w+, (\w+), SWIGLU", text)]
    assert [s[:2] for s in shapes] == [t[:2] for t in tiles.table()[0]]
    assert [s[2] for s in shapes] == ["1", "1", "2", "1", "kOnce"]


@pytest.mark.parametrize("tile,T,E,N,K,kind,act", tiles.SEVERAL)
def test_several_tiles(tile, T, E, N, K, kind, act):
    assert tiles.shape(T, E, N, K, act) == tile
    assert 2 <= tiles.most_of_workgroup(*tile, counts(T, E, N, K, kind), N, act) <= 4


@pytest.mark.parametrize("tile,T,E,N,K,kind,act,gather", tiles.MANY)
def test_many_tiles(tile, T, E, N, K, kind, act, gather):
    assert tiles.shape(T, E, N, K, act) == tile
    assert tiles.most_of_workgroup(*tile, counts(T, E, N, K, kind), N, act) > tiles.RING


def test_every_persistent_shape_is_there():
    for cases in (tiles.SEVERAL, tiles.MANY):
        assert {c[0] for c in cases} == {t[:2] for t in tiles.table()[0]} - {(32, 128)}
    wide = {(c[0], c[3] % 8 == 0) for c in tiles.SEVERAL}
    assert {(64, 256), (128, 256)} <= {c for c, w in wide if w} & {c for c, w in wide if not w}
