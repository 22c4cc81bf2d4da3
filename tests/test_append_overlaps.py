"""spec_verify_append refuses a cache that lies over what it reads while it writes
the cache, on the host: every call here returns before it launches anything."""

from __future__ import annotations

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_prompt_abi import append, rotary
from tests.test_serving_abi import P, cache

CACHE = {"k_pages": P[0], "v_pages": P[1], "k_scale": P[2], "v_scale": P[3], "k_tail": P[4], "v_tail": P[5]}


@pytest.mark.parametrize("name", CACHE)
@pytest.mark.parametrize("what", ["positions", "blocks", "lens", "freqs", "ids", "axes", "table", "positions_out", "blocks_out"])
def test_refuses_arguments_inside_the_cache(what, name):
    at = CACHE[name] + 16
    if what in ("freqs", "ids", "axes"):
        kw = dict(rot=rotary(**dict(dict(ids=P[32], num_axes=2, axes=P[31]), **{what: at})))
    elif what == "table":
        kw = dict(c=cache(block_table=at))
    else:
        kw = {what: at}
    assert append(**kw) == B.SV_ERR_ARG
