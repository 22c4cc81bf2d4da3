"""Waves of cache_append's kernels to a SIMD, which its registers leave: they hold
the cosines of a whole page, so that they go down with the page."""

from __future__ import annotations

import pytest

from tests.test_serving_resources import kernels  # noqa: F401  (a fixture)


@pytest.mark.parametrize("D, page, waves", [(64, 16, 5), (64, 32, 5), (64, 64, 5), (64, 128, 4), (64, 256, 2), (128, 16, 5),
                                            (128, 32, 5), (128, 64, 4), (128, 128, 2), (128, 256, 1)])
def test_waves_by_page(kernels, D, page, waves):  # noqa: F811
    mine = [v for k, v in kernels.items() if "cache_append_kernel" in k and f"Li{D}ELi{page}E" in k]
    assert len(mine) == 2
    for v in mine:
        assert int(v["Occupancy [waves/SIMD]"]) >= waves, v
        assert waves * int(v["LDS Size [bytes/block]"]) <= 160 * 1024
