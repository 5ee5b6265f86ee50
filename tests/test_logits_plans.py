"""The shapes that the GPU tests run for a tile of the 8-bit head's product still reach it, and together they reach all."""

from logits_plans import PLANS, TILES, plan


def test_shapes_reach_the_tiles_they_are_named_for(tmp_path):
    for shape, got in zip(PLANS, plan(list(PLANS), str(tmp_path))):
        assert got == PLANS[shape], (shape, got)


def test_every_tile_has_a_shape():
    assert {v[0] for v in PLANS.values()} == set(TILES)
    assert {v[1] for v in PLANS.values()} == set(TILES[2:])
    for side, names in ((0, TILES), (1, TILES[2:])):
        for t in names:   # a last block of k that is cut, for each
            assert any(v[side] == t and k[2] % 128 for k, v in PLANS.items()), t
