"""Whole serving steps: attention over the cache, logits from its output, adjusted, verified, committed, evicted,
step after step.  The reference follows the state from the accepted paths in float64."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R
from tests.test_gpu_attention import check as check_attention
from tests.test_gpu_attention import random_parents
from tests.test_gpu_commit import check as check_commit

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("kind, tree", [("e4m3", False), ("int8", True)])
def test_steps(kind, tree):
    B, T, H, Hkv, D, page, V, budget = 3, 7, 4, 2, 64, 16, 500, 3
    g = torch.Generator().manual_seed(5)
    cache = rsv.new_cache(B, B * 8, Hkv, D, page=page, max_blocks=8, max_new=T, kind=kind)
    cache.block_table.copy_(torch.randperm(B * 8, generator=g).view(B, 8))
    positions, blocks = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    totals = torch.zeros((B, 8), device="cuda")
    head = torch.randn((H * D, V), generator=g).cuda() * 0.3
    history = torch.zeros((B, 400), dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")       # one prompt token, the first root
    prompt = torch.ones(B, dtype=torch.int32, device="cuda")
    rep = torch.full((B,), 1.1, device="cuda")
    words = torch.full((2, (V + 31) // 32), -1, dtype=torch.int32)
    words[1, 3:] = 0                                             # a grammar that allows 96 tokens
    mask = words.cuda()
    temperature = torch.tensor([0.8, 0.0, 1.0], device="cuda")
    accepted = evicted = 0
    for step in range(40):
        before = dict(kind=kind, page=page, D=D, Hkv=Hkv, B=B, tail=cache.tail,
                      **{k: getattr(cache, "block_table" if k == "table" else k).cpu() for k in R.TENSORS},
                      positions=positions.cpu(), blocks=blocks.cpu())
        qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g).to(BF16)
        dev = qkv.cuda()
        parents = random_parents(step, B, T) if tree else None
        par = None if parents is None else parents.cuda()
        out, w = rsv.cache_attention(dev[:, :, :H], dev[:, :, H:H + Hkv], dev[:, :, H + Hkv:], cache, positions, blocks,
                                     parents=par, weights=True)
        check_attention(before, qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:], out, w, parents=parents)
        target = (out.float().reshape(B, T, H * D) @ head).to(BF16)
        draft = (target.float() + 0.5 * torch.randn(target.shape, generator=g).cuda()).to(BF16)
        # drafted tokens: the drafter's favourites at the parent, which are often the target's too
        source = draft.float().argsort(-1, descending=True)[:, :, :4]
        tokens = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        for c in range(1, T):
            p = par[:, c].long() if tree else torch.full((B,), c - 1, device="cuda")
            tokens[:, c] = source[torch.arange(B), p, c % 4 if tree else 0].int()
        rows = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
        rows[2] = 1
        ctl = dict(history=history, history_lens=lens, prompt_lens=prompt, repetition=rep, mask=mask, mask_rows=rows)
        uni = torch.rand((B, T), generator=g).cuda()
        if tree:
            adj = rsv.adjust_logits(target, tokens, parents=par, **ctl)
            dft = rsv.adjust_logits(draft, tokens, parents=par, **ctl)
            res, nodes, num = rsv.verify_tree(adj, dft, tokens, par, uni, temperature)
        else:
            chain = tokens[:, 1:].contiguous()
            adj = rsv.adjust_logits(target, chain, **ctl)
            dft = rsv.adjust_logits(draft[:, :T - 1], chain, **dict(ctl, mask_rows=rows[:, :T - 1].contiguous()))
            res, num = rsv.verify(adj, dft, chain, uni, temperature)
            nodes = None
        assert (res[2][:int(num[2]) + 1] < 96).all()             # the grammar held
        t0 = totals.cpu()
        outs = rsv.cache_commit(cache, dev[:, :, H:H + Hkv], dev[:, :, H + Hkv:], num, positions, blocks, nodes=nodes,
                                weights=w, totals=totals)
        check_commit(before, torch.stack([qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]], 2), num.cpu(), cache, outs,
                     None if nodes is None else nodes.cpu(), w.cpu(), t0)
        positions, blocks, totals = outs
        for b in range(B):
            n = int(num[b]) + 1
            history[b, int(lens[b]):int(lens[b]) + n] = res[b, :n]
        lens += num + 1
        accepted += int(num.sum())
        want = R.evict(cache.block_table.cpu(), totals.cpu(), blocks.cpu(), budget, 1, 1)
        _, totals, blocks, gone = rsv.cache_evict(cache.block_table, totals, blocks, budget, keep_first=1, keep_last=1,
                                                  table_out=cache.block_table, totals_out=totals, blocks_out=blocks)
        for x, y in zip((cache.block_table, totals, blocks, gone), want):
            np.testing.assert_array_equal(x.cpu().numpy(), y)
        evicted += int(gone.sum())
    assert accepted > 0 and evicted > 0 and int(blocks.max()) <= budget
