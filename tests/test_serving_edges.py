"""Argument checks of the operators around a verification step that lie at the
edges of what they take, on the host: every call here returns before it
launches anything."""

from __future__ import annotations

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_abi import OUT, P, WEIGHTS, adjust, attention, commit, evict


@pytest.mark.parametrize("width", [-1, 5])
def test_a_history_is_no_wider_than_its_rows_are_apart(width):
    assert adjust(c_repetition=P[3], c_history=P[5], c_history_lens=P[6], c_history_stride=4,
                  c_history_width=width) == B.SV_ERR_ARG


COUNTERS, TOTALS, NODES = 2 * 4, 2 * 10 * 4, 4 * (5 + 2)


@pytest.mark.parametrize("bad", [
    dict(totals_out=P[19]), dict(totals_out=P[19] + WEIGHTS - 4), dict(totals_out=P[19] + 4 - TOTALS),   # over weights
    dict(totals_out=P[6]), dict(totals_out=P[12] + 4), dict(totals_out=P[13]), dict(totals_out=P[14] + 4 - TOTALS),
    dict(totals_out=P[17] + NODES - 4), dict(totals_out=P[15]), dict(totals_out=P[16] - TOTALS + 4),
    dict(positions_out=P[6] + TOTALS - 4), dict(blocks_out=P[17] + NODES - 4), dict(positions_out=P[19]),
    dict(blocks_out=P[18] + 4)])
def test_commit_refuses_outputs_over_what_it_reads(bad):
    a = dict(nodes=P[17], stride=5, weights=P[19], totals=P[18], totals_out=P[20])
    assert commit(**dict(a, **bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(evicted=P[0]), dict(evicted=P[1] + 1600 - 4), dict(evicted=P[3] + 8), dict(evicted=P[4] - 12),
    dict(blocks_out=P[0] + 1596), dict(blocks_out=P[1]), dict(blocks_out=P[3] - 12), dict(blocks_out=P[4]),
    dict(totals_out=P[2] - 1596), dict(table_out=P[2])])
def test_evict_refuses_outputs_over_what_it_reads(bad):
    assert evict(**bad) == B.SV_ERR_ARG


PAGES, TAIL = 100 * 2 * 16 * 64, 2 * 32 * 2 * 64 * 2


@pytest.mark.parametrize("bad", [
    dict(out=P[20]), dict(out=P[20] + 16 - OUT), dict(weights=P[20] + 64), dict(weights=P[0] + PAGES - 4),
    dict(out=P[1]), dict(out=P[4] + TAIL - 16), dict(weights=P[5]), dict(weights=P[2] + 796), dict(out=P[3]),
    dict(out=P[6]), dict(weights=P[13] + 4), dict(weights=P[14] + 4 - WEIGHTS), dict(out=P[16], parents=P[16]),
    dict(weights=P[17], lens=P[17])])
def test_attention_refuses_outputs_over_any_input(bad):
    assert attention(**bad) == B.SV_ERR_ARG
