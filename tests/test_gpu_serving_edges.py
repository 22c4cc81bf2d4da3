"""Calls of the operators around a verification step that their documentation
allows and that lie at its edges."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import test_gpu_adjust_logits as A

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("first, width", [(0, 4), (3, 4), (5, 0), (2, 37)])
def test_lengths_beyond_a_view_of_a_wider_history(first, width):
    """Rows of the view lie 64 apart and are `width` long: lengths past that count what the view holds, no more."""
    B, P, V = 3, 4, 500
    logits, x = A.make(70, B, P, V, BF16, hist=40)
    wide = torch.randint(0, 60, (B, 64), dtype=torch.int32, generator=torch.Generator().manual_seed(71)).cuda()
    x["history"] = wide[:, first:first + width]
    x["history_lens"] = torch.tensor([64, width + 1, 2 ** 31 - 1], dtype=torch.int32).cuda()
    x["prompt_lens"] = None
    A.check(logits, x, rsv.adjust_logits(logits, **x))
