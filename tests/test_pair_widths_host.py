"""The widths of tiles that the host chooses, for the 76 CTA pairs of 152 SMs."""

import pytest

from optimizer_tcgen05_dw_gb300.build import build
from test_gpu_pair_widths import FORWARD, GRADIENT, PRODUCT, width_of


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()


@pytest.mark.parametrize("op,table,widths", [("forward", FORWARD, {128, 64, 32}), ("gradient", GRADIENT, {128, 64}),
                                             ("product", PRODUCT, {128, 64, 32})])
def test_the_tested_shapes_reach_every_width(op, table, widths):
    """Every width, of the kernels for up to 32 rows too, has a shape in the GPU tests."""
    for width, T, cols, _ in table:
        assert width_of(op, T, cols, 76) == width, (op, T, cols)
    assert {w for w, T, _, _ in table if T > 32} == widths
    if op != "gradient":
        assert {w for w, T, _, _ in table if T <= 32} == widths
