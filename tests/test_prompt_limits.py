"""Launches of 2^32 work-items and more are refused before anything runs, on the
host: sizes at the border of what the calls that bring prompts in and draw
tokens take.  Every call here is a size query or is refused."""

from __future__ import annotations

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_sample_abi import call
from tests.test_serving_abi import P


@pytest.mark.parametrize("dtype, part", [(B.SV_BF16, 8192), (B.SV_F32, 4096)])
def test_truncate_counts_the_work_groups_of_its_last_kernel(dtype, part):
    """It has one to `part` logits (and a lead of one vector), the first one to twice as many."""
    rows, V = 1 << 23, part + 1
    one = dict(P=1, V=V, row=V, stride=V, out_row=V, out_stride=V, dtype=dtype)
    rc, n = call("truncate", ws=None, B=rows - 1, **one)
    assert rc == B.SV_OK and n > 0
    rc, _ = call("truncate", ws=None, B=rows, **one)
    assert rc == B.SV_ERR_UNSUPPORTED
    assert call("truncate", B=rows, **dict(one, out=P[0])) == B.SV_ERR_UNSUPPORTED   # in place
    rc, n = call("sample", ws=None, B=rows, **{k: one[k] for k in ("P", "V", "row", "stride", "dtype")})
    assert rc == B.SV_OK and n > 0
