"""Rows that answer one prompt, as a program serves them: the prompt is
appended once, the rows share its pages, and each step rotates, attends, cuts
the logits, draws drafts, verifies and commits.  Every call is compared with
its reference, on the state that the calls before it left."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R
from tests import rotary_ref as RR
from tests import sample_ref as S
from tests.test_gpu_commit import check as check_commit
from tests.test_gpu_prefix import check as check_attention
from tests.test_gpu_rotate import freqs_of, near

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def snapshot(cache, positions, blocks, kind):
    return dict(kind=kind, page=cache.page, D=cache.D, Hkv=cache.Hkv, B=cache.B, tail=cache.tail,
                **{k: getattr(cache, "block_table" if k == "table" else k).cpu() for k in R.TENSORS},
                positions=positions.cpu(), blocks=blocks.cpu())


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_answers_to_one_prompt(kind):
    B, K, H, Hkv, D, page, V, most = 4, 3, 4, 2, 64, 16, 700, 8
    T, L = K + 1, 93                                         # a prompt of five blocks and 13 tokens
    g = torch.Generator().manual_seed(3)
    cache = rsv.new_cache(B + 1, B * most + 8, Hkv, D, page=page, max_blocks=most, max_new=T, kind=kind)
    cache.block_table.copy_(torch.randperm(B * most + 8, generator=g)[:(B + 1) * most].view(B + 1, most))
    freqs = freqs_of(D).cuda()
    positions, blocks = (torch.zeros(B + 1, dtype=torch.int32, device="cuda") for _ in range(2))

    # The prompt enters by the last row; the others append nothing.
    prompt = torch.randn((B + 1, L, 2, Hkv, D), generator=g).to(BF16)
    lens = torch.zeros(B + 1, dtype=torch.int32)
    lens[B] = L
    before = snapshot(cache, positions, blocks, kind)
    dev = prompt.cuda()
    rotated = torch.zeros((B + 1, L, Hkv, D), dtype=BF16, device="cuda")
    outs = rsv.cache_append(cache, dev[:, :, 0], dev[:, :, 1], positions, blocks, lens=lens.cuda(), freqs=freqs, k_out=rotated)
    at = torch.arange(L)[None, None].expand(1, B + 1, L)
    near(rotated[B:], prompt[B:, :, 0], freqs.cpu(), False, at[:, :1], None)
    kv = torch.stack([rotated.cpu(), prompt[:, :, 1]], 2)
    check_commit(before, kv, lens - 1, cache, outs)
    positions, blocks = outs
    assert positions.tolist() == [0] * B + [L] and blocks.tolist() == [0] * B + [L // page]

    # Its pages become the others' prefix, what is left of it their tail.
    n = L // page
    prefix = dict(prefix_table=cache.block_table[B:, :n].contiguous(),
                  prefix_blocks=torch.tensor([n], dtype=torch.int32, device="cuda"),
                  prefix_starts=torch.tensor([0, B], dtype=torch.int32, device="cuda"))
    cache.k_tail[:B] = cache.k_tail[B]
    cache.v_tail[:B] = cache.v_tail[B]
    positions[:B] = L
    idle = torch.tensor([T] * B + [0], dtype=torch.int32)    # the prompt's own row rests

    head = torch.randn((H * D, V), generator=g).cuda()
    temperature = torch.full((B + 1,), 0.9, device="cuda")
    top_k = torch.tensor([20, 0, 5, 40, 0], dtype=torch.int32, device="cuda")
    top_p = torch.tensor([0.9, 0.95, 1.0, 0.5, 1.0], device="cuda")
    accepted = 0
    for step in range(12):
        before = snapshot(cache, positions, blocks, kind)
        qkv = torch.randn((B + 1, T, H + 2 * Hkv, D), generator=g).to(BF16)
        x = qkv.cuda()
        q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
        rsv.rotate_tokens(q, k, freqs, positions, query_lens=idle.cuda(), q_out=q, k_out=k)
        ids = RR.token_positions(before["positions"], T)[None]
        near(q[:B].contiguous(), qkv[:B, :, :H], freqs.cpu(), False, ids[:, :B], None)
        near(k[:B].contiguous(), qkv[:B, :, H:H + Hkv], freqs.cpu(), False, ids[:, :B], None)
        out, w = rsv.cache_attention(q, k, v, cache, positions, blocks, query_lens=idle.cuda(), weights=True, **prefix)
        whole = dict(before, table=torch.cat([before["table"][B:, :n].expand(B + 1, n), before["table"]], 1),
                     blocks=before["blocks"] + torch.tensor([n] * B + [0], dtype=torch.int32))
        whole["table"][B, :most] = before["table"][B]
        check_attention(whole, [n] * B + [0], most, q.cpu(), k.cpu(), v.cpu(), out, w, query_lens=idle)

        target = (out.float().reshape(B + 1, T, H * D) @ head).to(BF16)
        draft = (target[:, :K].float() + 0.5 * torch.randn((B + 1, K, V), generator=g).cuda()).to(BF16)
        target, draft = (rsv.truncate_logits(z, temperature, top_k=top_k, top_p=top_p) for z in (target, draft))
        u = torch.rand((B + 1, K, 1), generator=g)
        tokens, logprobs = rsv.sample_tokens(draft, u.cuda(), temperature, top_k=top_k, top_p=top_p, logprobs=True)
        for b in range(B):
            for i in range(K):
                row = draft[b, i].double().cpu().numpy()
                ids_, weights = S.kept(row, float(temperature[b]), int(top_k[b]), float(top_p[b]))
                want = S.draw(ids_, weights, float(u[b, i, 0]))
                assert int(tokens[b, i, 0]) == want[0] and abs(float(logprobs[b, i, 0]) - want[1]) < 1e-5
        uni = torch.rand((B + 1, T), generator=g).cuda()
        res, num = rsv.verify(target, draft, tokens[:, :, 0].contiguous(), uni, temperature)
        for b in range(B):   # nothing that the cut left out is emitted
            at_ = int(num[b])
            assert float(target[b, at_, int(res[b, at_])]) > -float("inf")
        num[B] = -1
        outs = rsv.cache_commit(cache, k, v, num, positions, blocks)
        check_commit(before, torch.stack([k.cpu(), v.cpu()], 2), num.cpu(), cache, outs)
        positions, blocks = outs
        accepted += int(num[:B].sum())
    assert accepted > 0 and int(blocks[:B].max()) > 0 and int(blocks[B]) == n
