"""cache_attention's prefix arguments as a serving program changes them from call
to call: tables that grow, and one workspace for all of them."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding
from tests import cache_ref as R
from tests.test_gpu_attention import make_qkv, views
from tests.test_gpu_prefix import check, shared_state

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


RANGES = {  # starts -> the prefix of each of five rows, -1: none
    (0, 2, 5): [0, 0, 1, 1, 1], (5, -3, 9): [1] * 5, (3, 1, 2): [-1, 1, -1, -1, -1], (-2 ** 31, 2 ** 31 - 1, 0): [0] * 5,
    (2, 2, 4): [-1, -1, 1, 1, -1], (9, 9, 9): [-1] * 5, (3, 4, 1): [-1, -1, -1, 0, -1], (-7, -7, 2): [1, 1, -1, -1, -1]}


@pytest.mark.parametrize("lengths", [(9, 5), (-1, 10 ** 9), (-2 ** 31, 2 ** 31 - 1), (0, 3)])
@pytest.mark.parametrize("starts", RANGES, ids=str)
def test_ranges_and_lengths_of_any_kind(starts, lengths):
    """What lies in no range goes without a prefix, lengths count as what the table holds, and nothing is written
    beside the outputs and the workspace."""
    rows, prefix, _, _ = shared_state(33, [20, 300, 0, 45, 7], [9, 5], [0, 2, 5], Hkv=2, D=64, page=16, kind="e4m3")
    cache, positions, blocks = R.to_gpu(rows)
    qkv = make_qkv(34, 5, 3, 8, 2, 64)
    table, width = prefix["prefix_table"], prefix["prefix_table"].shape[1]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n = rsv.attention_workspace_bytes(cache, 3, 8, weights=True, prefix=(2, width))
    around = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    around[256:256 + n] = 0
    outs = torch.full((7, 3, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    masses = torch.full((7, 3, cache.max_blocks), 7.0, device="cuda")
    rsv.cache_attention(*views(qkv.cuda(), 8, 2), cache, positions, blocks, prefix_table=table.cuda(),
                        prefix_blocks=i32(lengths), prefix_starts=i32(starts), out=outs[1:6], weights=masses[1:6],
                        workspace=around[256:256 + n])
    assert (around[:256] == 0xA5).all() and (around[256 + n:] == 0xA5).all()
    for t in (outs, masses):
        assert (t[0] == 7).all() and (t[6] == 7).all()
    # the rows as if their prefixes' pages stood in their own tables
    before = [0 if i < 0 else min(max(lengths[i], 0), width) for i in RANGES[starts]]
    own = rows["table"].shape[1]
    whole = dict(rows, table=torch.full((5, width + own), -1, dtype=torch.int32), blocks=rows["blocks"] + torch.tensor(before))
    for b, i in enumerate(RANGES[starts]):
        whole["table"][b, :before[b]] = table[i, :before[b]]
        whole["table"][b, before[b]:before[b] + own] = rows["table"][b]
    check(whole, before, own, *views(qkv, 8, 2), outs[1:6], masses[1:6])
