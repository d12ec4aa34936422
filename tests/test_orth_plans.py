"""The update's GPU tests reach every kernel that its cost model can choose, whatever the table of measured times says."""
from _orth import SIZES, plans


def test_every_tile_shape_is_reached():
    rows, shapes = plans(tuple(SIZES))
    every = set(range(shapes))
    assert {g for g, parts, _, _ in rows if parts == 1} == every
    assert {g for g, parts, _, _ in rows if parts > 1} == every
    assert {p for _, _, p, _ in rows} == every
    assert {x for _, _, _, x in rows} == every
