"""The shapes that the GPU tests run for a path of the vocabulary head still reach it, and together they reach all."""

from head_plans import PLANS, plan


def test_shapes_reach_the_paths_they_are_named_for(tmp_path):
    for shape, got in zip(PLANS, plan(list(PLANS), str(tmp_path))):
        assert got == PLANS[shape], (shape, got)


def test_every_path_has_a_shape():
    bf16 = [v for k, v in PLANS.items() if k[3] == "bf16"]
    f32 = [v for k, v in PLANS.items() if k[3] == "f32"]
    tiles = {"big", "mid", "thin", "deep", "small"}
    for use in (0, 1):   # the logits' products
        assert {t for v in bf16 for t in v[use].split("+")} == tiles | {"A"}
        assert {v[use] for v in f32} == {"thin", "small"}
    assert {v[2] for v in bf16} == {"big", "mid", "A+mid", "B+mid"} and {v[2] for v in f32} == {"thin", "small"}
    acc = {v[3] for v in bf16}
    assert {("thin", False, True), ("mid", True, True), ("big", True, True), ("big", False, True)} <= acc
    assert any(v[3] == ("big", True, True) and v[4] > 1 for v in bf16)   # whole and shared tiles over two pieces
    assert {("small", True, True), ("thin", True, True)} <= {v[3] for v in f32}
    # last steps of 128 bytes of k, whole and cut, for both kinds of deep products
    rest = {k[2] * 2 % 128 != 0 for k, v in PLANS.items() if v[0] == "deep"}
    assert rest == {True, False}
