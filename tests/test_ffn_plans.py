"""The kernels that the GPU tests of the feed-forward operators mean to run are
the ones the plan gives their cases (no GPU)."""
import pytest

import ffn_plans

pytestmark = pytest.mark.skipif(not ffn_plans.have_compiler, reason="needs g++")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return ffn_plans.printer(tmp_path_factory.mktemp("plans"))


def test_linear_cases_take_their_tile_shapes(exe):
    cases = {**ffn_plans.TILES, **ffn_plans.SPLIT_TILES, **ffn_plans.WHOLE_TILES}
    for aligned in (0, 1):
        got = ffn_plans.plans(exe, [f"{n} {m} {k} {int(g)} 1 {aligned}" for n, m, k, g in cases])
        for (n, m, k, g), want, plan in zip(cases, cases.values(), got):
            copied = 0 if aligned else 2 * n * k
            assert plan == f"{want} {copied}", f"{n} x ({m} x {k}), gated {g}"


def test_every_tile_shape_is_among_them(exe):
    seen = {(g, want.split()[1]) for (_, _, _, g), want in ffn_plans.TILES.items()}
    assert seen == {(False, s) for s in ("64x32", "64x64", "128x64", "128x128", "256x128", "256x256")} | \
        {(True, s) for s in ("64x32", "64x64", "64x128", "128x128", "128x256")}


def test_moe_cases_take_their_kernels(exe):
    """Shapes of the routing tests: the choice by the up product's workgroups, with a small
    router and with a large one, and on its own."""
    from test_gpu_ffn_routing import SHAPES

    got = ffn_plans.plans(exe, [f"moe {t} {e} {k} {h} {i}" for t, e, k, h, i in SHAPES])
    assert got == ["few 1", "few 0", "sorted 1", "sorted 1"]
    assert SHAPES[2][0] <= 16 < SHAPES[3][0]   # by one workgroup, and by one per four tokens
