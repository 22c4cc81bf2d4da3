"""cache_attention under graph capture with a workspace of the graph's own."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import serving_ops
from tests import cache_ref as R
from tests.test_gpu_attention import make_qkv, random_parents, views

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H, Hkv, D, T, tree", [(4, 2, 64, 3, False), (16, 2, 128, 13, True), (7, 1, 64, 5, False),
                                                (8, 4, 64, 33, True)])
def test_a_graph_clears_the_counters_alone(H, Hkv, D, T, tree, monkeypatch):
    """Partial sums and masses are written before they are read, so a replay need not clear them: only the counters'
    bytes are set in the graph, and replays over a workspace of rubbish give the eager results."""
    B = 3
    s = R.random_state(90, B=B, Hkv=Hkv, D=D, page=16, kind="e4m3", contexts=[3000, 0, 700])
    qkv = make_qkv(91, B, T, H, Hkv, D).cuda()
    q, kn, vn = views(qkv, H, Hkv)
    parents = random_parents(92, B, T).cuda() if tree else None
    cache, positions, blocks = R.to_gpu(s)
    want = [t.clone() for t in rsv.cache_attention(q, kn, vn, cache, positions, blocks, parents=parents, weights=True)]
    need = rsv.attention_workspace_bytes(cache, T, H, tree=tree, weights=True)
    counters = 4 * B * Hkv * -(-(T * H // Hkv) // 16)
    assert counters < need // 16
    made = []

    def rubbish(*size, **kw):
        t = torch.full(size, 0xA5, **kw) if kw.get("dtype") is torch.uint8 else real_empty(*size, **kw)
        if kw.get("dtype") is torch.uint8:
            made.append(t)
        return t

    real_empty, real_zeros = torch.empty, torch.zeros

    def no_large_zeros(*size, **kw):
        assert kw.get("dtype") is not torch.uint8, "the whole workspace is cleared in the graph"
        return real_zeros(*size, **kw)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    monkeypatch.setattr(serving_ops.torch, "empty", rubbish)
    monkeypatch.setattr(serving_ops.torch, "zeros", no_large_zeros)
    with torch.cuda.graph(graph):
        out, w = rsv.cache_attention(q, kn, vn, cache, positions, blocks, parents=parents, weights=True)
    monkeypatch.undo()
    assert len(made) == 1 and made[0].numel() == need
    for i in range(4):
        out.zero_()
        w.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(w, want[1])
        eager = rsv.cache_attention(q, kn, vn, cache, positions, blocks, parents=parents, weights=True)
        assert torch.equal(eager[0], want[0]) and torch.equal(eager[1], want[1])


def test_a_given_workspace_needs_no_more_than_its_counters_cleared():
    B, T, H, Hkv, D = 2, 6, 8, 2, 128
    s = R.random_state(93, B=B, Hkv=Hkv, D=D, page=64, kind="int8", contexts=[5000, 90])
    q, kn, vn = views(make_qkv(94, B, T, H, Hkv, D).cuda(), H, Hkv)
    cache, positions, blocks = R.to_gpu(s)
    want = rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=True)
    ws = torch.full((rsv.attention_workspace_bytes(cache, T, H, weights=True),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4 * B * Hkv * -(-(T * H // Hkv) // 16)] = 0
    for _ in range(3):
        got = rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=True, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
