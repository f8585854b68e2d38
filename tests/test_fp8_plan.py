"""Which kernel takes a product of 8-bit matrices (host logic, no GPU), and that the shapes the GPU tests name for
the many-row kernel reach it."""
import ctypes

import pytest

from lut_dequant_gemv_b200 import binding as B
from lut_dequant_gemv_b200 import build as build_mod
from test_gpu_fp8_many import SHAPES


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("width,m,n,k", SHAPES)
def test_shapes_of_the_many_row_tests_reach_it(width, m, n, k):
    assert B.sqz_fp8_plan_query(m, n, k) == dict(many_rows=1, tile_rows=256, tile_cols=width, splits=1)


def test_every_width_wraps_its_scales_and_its_tiles():
    """Between them the shapes have, at every width, more than 16 blocks of K (the scales come 16 at a time, in two
    buffers), a last tile that is partial, and once more than 32 blocks; and somewhere more tiles than pairs of SMs."""
    for width in (64, 128, 160, 192, 256):
        mine = [(m, n, k) for w, m, n, k in SHAPES if w == width]
        assert any(k > 2048 for _, _, k in mine) and any(n % width for _, n, _ in mine), width
    assert any(k > 4096 for _, _, _, k in SHAPES)
    assert any(-(-m // 256) * -(-n // w) > 74 for w, m, n, _ in SHAPES)


def test_few_rows_share_k_within_a_cluster():
    for m in (1, 2, 16, 17, 32, 33, 64):
        for n in (1, 128, 4096, 13824):
            for k in (1, 128, 129, 4096, 13824):
                p = B.sqz_fp8_plan_query(m, n, k)
                assert p["many_rows"] == 0 and p["tile_rows"] == (16 if m <= 16 else 32 if m <= 32 else 64)
                assert 1 <= p["splits"] <= min(8, -(-k // 128))


def test_few_rows_of_very_wide_matrices():
    """More blocks of W's rows than a grid has in its second dimension go to the many-row kernel."""
    assert B.sqz_fp8_plan_query(1, 65535 * 128, 128)["many_rows"] == 0
    assert B.sqz_fp8_plan_query(1, 65535 * 128 + 1, 128)["many_rows"] == 1


def test_the_largest_sizes_have_a_plan():
    top = 2 ** 31 - 257
    for m in (1, 300, top):
        for n in (1, 300, top):
            for k in (1, top):
                p = B.sqz_fp8_plan_query(m, n, k)
                assert p["splits"] >= 1 and p["tile_rows"] >= 16
                if not p["many_rows"]:  # a grid's third dimension has room
                    assert -(-m // p["tile_rows"]) <= 65535


@pytest.mark.parametrize("bad", [(0, 1, 1, 148), (1, 0, 1, 148), (1, 1, 0, 148), (2 ** 31 - 256, 1, 1, 148), (1, 1, 1, 1)])
def test_refusals(lib, bad):
    out = B.sqz_fp8_plan_info()
    assert lib.sqz_fp8_plan_query(*bad, ctypes.byref(out)) == B.SQZ_ERR_INVALID_ARG
    assert lib.sqz_fp8_plan_query(1, 1, 1, 148, None) == B.SQZ_ERR_INVALID_ARG
