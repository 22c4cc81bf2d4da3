"""Register and LDS budgets of the operators around a verification step, from
the compiler's resource report that each build writes next to the library.

Two work-groups of the attention kernel share a CU: its waves must fit two to
a SIMD and its LDS twice into 160 KB, or the runs that it is cut into no
longer fill the chip at once.
"""

from __future__ import annotations

import os
import re

import pytest

from rejection_sampling_verifier_amd import build as BUILD


@pytest.fixture(scope="module")
def kernels():
    sources = [os.path.join(BUILD.SERVING_DIR, f) for f in os.listdir(BUILD.SERVING_DIR)]
    if (not os.path.exists(BUILD.RESOURCES)
            or os.path.getmtime(BUILD.RESOURCES) < max(os.path.getmtime(f) for f in sources)):
        pytest.skip("no resource report of these sources: build first")
    found, cur = {}, None
    for line in open(BUILD.RESOURCES).read().splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            cur = found.setdefault(m.group(1), {})
            continue
        m = re.search(r"remark:\s+([A-Za-z][A-Za-z /\[\]]*?): (\S+) \[-Rpass", line)
        if m and cur is not None:
            cur[m.group(1).strip()] = m.group(2)
    return found


@pytest.mark.parametrize("name, variants", [("cache_attention_kernel", 20), ("attention_weights_kernel", 3),
                                            ("adjust_logits_kernel", 2), ("cache_commit_kernel", 20),
                                            ("cache_evict_kernel", 6), ("cache_evict_long_kernel", 1)])
def test_no_kernel_uses_scratch(kernels, name, variants):
    mine = {k: v for k, v in kernels.items() if name in k}
    assert len(mine) == variants, sorted(mine)
    for k, v in mine.items():
        assert int(v["VGPRs Spill"]) == 0 and int(v["ScratchSize [bytes/lane]"]) == 0, (k, v)


def test_two_attention_work_groups_to_a_cu(kernels):
    for k, v in kernels.items():
        if "cache_attention_kernel" in k:
            assert int(v["Occupancy [waves/SIMD]"]) == 2, (k, v)
            assert 2 * int(v["LDS Size [bytes/block]"]) <= 160 * 1024, (k, v)
