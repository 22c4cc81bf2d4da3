"""cache_attention's prefix arguments as a serving program changes them from call
to call: tables that grow, and one workspace for all of them."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding
from tests import cache_ref as R
from tests.test_gpu_attention import make_qkv, views
from tests.test_gpu_prefix import shared_state

pytestmark = pytest.mark.gpu


def test_tables_of_any_width_share_a_workspace():
    rows, prefix, _, _ = shared_state(31, [20, 300, 0, 45], [9, 5], [0, 2, 4], Hkv=2, D=64, page=16, kind="e4m3")
    cache, positions, blocks = R.to_gpu(rows)
    qkv = make_qkv(32, 4, 3, 8, 2, 64).cuda()
    dev = {k: v.cuda() for k, v in prefix.items()}

    def call(width, count=2, **kw):
        table = torch.full((count, width), -1, dtype=torch.int32, device="cuda")
        n = min(width, 9)
        table[:2, :n] = dev["prefix_table"][:, :n]
        at = torch.cat([dev["prefix_starts"], dev["prefix_starts"][-1:].expand(count - 2)])
        b = torch.zeros(count, dtype=torch.int32, device="cuda")
        b[:2] = dev["prefix_blocks"].clamp(max=width)
        return rsv.cache_attention(*views(qkv, 8, 2), cache, positions, blocks, weights=True, prefix_table=table,
                                   prefix_blocks=b, prefix_starts=at.contiguous(), **kw)
    shapes = [(w, c) for w in (1, 3, 9, 10, 33, 70, 200, 2000, 65536) for c in (2, 5)]
    fresh = {s: call(*s, workspace=rsv.new_attention_workspace(cache, 3, 8, weights=True, prefix=(s[1], s[0]))) for s in shapes}
    binding.release_workspaces()
    held = set()
    for s in shapes + shapes[::-1]:
        out, w = call(*s)
        assert torch.equal(out, fresh[s][0]) and torch.equal(w, fresh[s][1]), s
        held.update((k, shape, t.data_ptr()) for k, per in binding._WS_CACHE.items() for shape, t in per.items())
    assert len(held) == 1, held
    # and one given workspace serves them too, the smallest first, and calls without a prefix between them
    ws = rsv.new_attention_workspace(cache, 3, 8, weights=True, prefix=(1, 65536))
    plain = rsv.cache_attention(*views(qkv, 8, 2), cache, positions, blocks, weights=True)
    for s in shapes:
        out, w = call(*s, workspace=ws)
        assert torch.equal(out, fresh[s][0]) and torch.equal(w, fresh[s][1]), s
        out, w = rsv.cache_attention(*views(qkv, 8, 2), cache, positions, blocks, weights=True, workspace=ws)
        assert torch.equal(out, plain[0]) and torch.equal(w, plain[1])
