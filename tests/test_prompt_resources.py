"""Register and LDS budgets of the operators that bring a prompt in and draw
tokens, from the compiler's resource report that each build writes."""

from __future__ import annotations

import pytest

from tests.test_serving_resources import kernels  # noqa: F401  (a fixture)


@pytest.mark.parametrize("name, variants", [("rotate_kernel", 2), ("cache_append_kernel", 20), ("append_counters_kernel", 1),
                                            ("sample_stats_kernel", 4), ("sample_row_kernel", 4), ("truncate_kernel", 4),
                                            ("prefix_attention_kernel", 8), ("prefix_join_kernel", 4)])
def test_no_kernel_uses_scratch(kernels, name, variants):  # noqa: F811
    mine = {k: v for k, v in kernels.items() if name in k}
    assert len(mine) == variants, sorted(mine)
    for k, v in mine.items():
        assert int(v["VGPRs Spill"]) == 0 and int(v["ScratchSize [bytes/lane]"]) == 0, (k, v)


@pytest.mark.parametrize("name, waves", [("prefix_attention_kernel", 2), ("sample_stats_kernel", 4), ("sample_row_kernel", 3)])
def test_waves_that_the_kernels_are_sized_for(kernels, name, waves):  # noqa: F811
    for k, v in kernels.items():
        if name in k:
            assert int(v["Occupancy [waves/SIMD]"]) >= waves, (k, v)
            assert waves * int(v["LDS Size [bytes/block]"]) <= 160 * 1024, (k, v)
