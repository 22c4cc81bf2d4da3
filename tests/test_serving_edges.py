"""Argument checks of the operators around a verification step that lie at the
edges of what they take, on the host: every call here returns before it
launches anything."""

from __future__ import annotations

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_abi import P, adjust


@pytest.mark.parametrize("width", [-1, 5])
def test_a_history_is_no_wider_than_its_rows_are_apart(width):
    assert adjust(c_repetition=P[3], c_history=P[5], c_history_lens=P[6], c_history_stride=4,
                  c_history_width=width) == B.SV_ERR_ARG
