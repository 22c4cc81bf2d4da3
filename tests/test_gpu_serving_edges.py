"""Calls of the operators around a verification step that their documentation
allows and that lie at its edges."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R
from tests import test_gpu_adjust_logits as A
from tests import test_gpu_attention as AT

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


def last_entries(ids, values, V):
    """Each token's last entry, by numpy's own order of assignment."""
    out = torch.zeros(V, dtype=torch.float64)
    seen = torch.zeros(V, dtype=torch.bool)
    for x, v in zip(ids.tolist(), values.tolist()):
        if 0 <= x < V:
            out[x], seen[x] = v, True
    return out, seen


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("V, entries, spread", [(9000, 1500, 4000), (9000, 2048, 9000), (9000, 2049, 2049),
                                                (9000, 9000, 9000), (4099, 20000, 4099), (5003, 3000, 7)])
def test_dense_biases(V, entries, spread, dtype):
    """Many biased ids side by side, and repeated ones: the last entry of each counts."""
    g = torch.Generator().manual_seed(72)
    B, P = 2, 5
    first = (V - spread) // 2
    ids = first + torch.randint(0, spread, (B, entries), generator=g, dtype=torch.int32)
    if entries == V:
        ids = torch.stack([torch.randperm(V, generator=g, dtype=torch.int32) for _ in range(B)])
    values = torch.randn((B, entries), generator=g)
    lens = torch.tensor([entries, entries - 700], dtype=torch.int32)
    logits = torch.randn((B, P, V), generator=g).to(dtype)
    got = rsv.adjust_logits(logits.cuda(), bias_ids=ids.cuda(), bias_values=values.cuda(), bias_lens=lens.cuda()).cpu()
    inplace = logits.cuda()
    rsv.adjust_logits(inplace, bias_ids=ids.cuda(), bias_values=values.cuda(), bias_lens=lens.cuda(), out=inplace)
    assert torch.equal(inplace.cpu(), got)
    for b in range(B):
        add, seen = last_entries(ids[b, :lens[b]], values[b, :lens[b]], V)
        ref = logits[b].double() + add
        # one float32 sum, 2^-24 of it, and the output's half step
        tol = (ref.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -24)) * (1 + 2.0 ** -20)
        assert ((got[b].double() - ref).abs() <= tol)[:, seen].all()
        assert torch.equal(got[b][:, ~seen], logits[b][:, ~seen])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("dtype, word, bits", [(BF16, torch.int16, 0x7F81), (torch.float32, torch.int32, 0x7F800001)])
def test_listed_logits_that_nothing_applies_to_keep_their_bits(dtype, word, bits, inplace):
    """A drafted token before its own position, and a prompt token without a repetition penalty: signalling NaN."""
    B, P, V = 1, 4, 300
    logits = torch.randn((B, P, V), generator=torch.Generator().manual_seed(73)).to(dtype)
    logits.view(word)[..., [5, 9, 40]] = bits
    want = logits.clone()
    logits = logits.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = rsv.adjust_logits(logits, i32([[7, 5, 9]]), history=i32([[40, 41]]), history_lens=i32([2]), prompt_lens=i32([2]),
                            presence=torch.ones(1, device="cuda"), out=logits if inplace else None).cpu()
    same = torch.ones((B, P, V), dtype=torch.bool)
    for i, t in ((1, 7), (2, 7), (2, 5), (3, 7), (3, 5), (3, 9)):
        same[0, i, t] = False
        assert float(want[0, i, t]) - 1 == pytest.approx(float(got[0, i, t]), rel=2 ** -7, nan_ok=True)
    assert torch.equal(got.view(word)[same], want.view(word)[same])


def test_eviction_counts_past_32_bits_and_below_zero():
    """A budget of 2^32 is no budget of 0."""
    i32 = dict(dtype=torch.int32, device="cuda")
    table, totals, blocks = torch.arange(12, **i32).view(2, 6), torch.rand((2, 6), device="cuda"), torch.tensor([6, 4], **i32)
    for kw in (dict(budget=2 ** 32), dict(budget=2 ** 63), dict(budget=2, keep_first=2 ** 32), dict(budget=0, keep_last=2 ** 40)):
        t, w, n, gone = rsv.cache_evict(table, totals, blocks, **kw)
        assert torch.equal(t, table) and torch.equal(n, blocks) and not gone.any()
        assert torch.equal(w[0], totals[0]) and torch.equal(w[1, :4], totals[1, :4])
    assert rsv.cache_evict(table, totals, blocks, 3, keep_first=2 ** 31 - 1)[3].tolist() == [0, 0]
    for kw in (dict(budget=-1), dict(budget=-2 ** 32), dict(budget=1, keep_first=-5), dict(budget=1, keep_last=-2 ** 33)):
        with pytest.raises(rsv.SpecVerifyError):
            rsv.cache_evict(table, totals, blocks, **kw)
    with pytest.raises(TypeError):
        rsv.cache_evict(table, totals, blocks, 2.5)


def test_a_cache_does_not_lose_its_tensors():
    cache = rsv.new_cache(1, 2, 1, 64, page=16)
    for name in ("block_table", "k_pages", "_c"):
        with pytest.raises(AttributeError):
            delattr(cache, name)


def test_more_rows_than_threads_with_several_row_tiles():
    """300 rows, several to a thread, each of up to three tiles of queries, some idle."""
    AT.case(74, [(29 * b) % 90 for b in range(300)], 33, 4, 2, 128, 32, "int8", tree=True,
            query_lens=[(11 * b) % 35 - 1 for b in range(300)])


@pytest.mark.parametrize("H, T", [(520, 3), (1040, 40)])
def test_more_heads_than_work_groups(H, T):
    """One run holds a whole line: the chip is filled by the heads alone."""
    AT.case(75, [100, 0, 33], T, H, 520, 64, 16, "e4m3")


def test_two_streams_at_once():
    """Calls without a workspace on two streams have one each."""
    B, T, H, Hkv, D = 4, 5, 8, 2, 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for i in range(2):
        s = R.random_state(76 + i, B=B, Hkv=Hkv, D=D, page=64, kind="e4m3", contexts=[6000, 40, 3000, 900 * i],
                           max_blocks=100)
        cache, positions, blocks = R.to_gpu(s)
        q, kn, vn = AT.views(AT.make_qkv(78 + i, B, T, H, Hkv, D).cuda(), H, Hkv)
        want = rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=True)
        jobs.append((q, kn, vn, cache, positions, blocks, want))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (stream, job) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(stream):
                got[i].append(rsv.cache_attention(*job[:6], weights=True))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for out, w in got[i]:
            assert torch.equal(out, job[6][0]) and torch.equal(w, job[6][1])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_whole_step_captured_and_replayed(kind):
    """Attention, controls, verification, commit and eviction in one graph that advances its state in place; each
    replay against the eager calls on a copy of the state."""
    B, T, H, Hkv, D, page, V, most = 3, 5, 4, 2, 64, 16, 700, 12
    g = torch.Generator().manual_seed(79)

    def state():
        cache = rsv.new_cache(B, B * most, Hkv, D, page=page, max_blocks=most, max_new=T, kind=kind)
        cache.block_table.copy_(torch.arange(B * most, dtype=torch.int32).view(B, most))
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(cache=cache, positions=z(B), blocks=z(B), totals=torch.zeros((B, most), device="cuda"))

    inputs = dict(qkv=torch.zeros((B, T, H + 2 * Hkv, D), dtype=BF16, device="cuda"),
                  draft=torch.zeros((B, T - 1, V), dtype=BF16, device="cuda"),
                  tokens=torch.zeros((B, T - 1), dtype=torch.int32, device="cuda"),
                  uniforms=torch.zeros((B, T), device="cuda"))
    head = (torch.randn((H * D, V), generator=g) * 0.02).cuda()
    presence, temperature = torch.full((B,), 0.3, device="cuda"), torch.full((B,), 1.0, device="cuda")

    def step(s, x):
        q, kn, vn = x["qkv"][:, :, :H], x["qkv"][:, :, H:H + Hkv], x["qkv"][:, :, H + Hkv:]
        out, w = rsv.cache_attention(q, kn, vn, s["cache"], s["positions"], s["blocks"], weights=True)
        target = (out.reshape(B, T, H * D).float() @ head).to(BF16)
        rsv.adjust_logits(target, x["tokens"], presence=presence, out=target)
        res, num = rsv.verify(target, x["draft"], x["tokens"], x["uniforms"], temperature)
        rsv.cache_commit(s["cache"], kn, vn, num, s["positions"], s["blocks"], weights=w, totals=s["totals"],
                         positions_out=s["positions"], blocks_out=s["blocks"], totals_out=s["totals"])
        table = s["cache"].block_table
        gone = rsv.cache_evict(table, s["totals"], s["blocks"], 3, keep_first=1, keep_last=1, table_out=table,
                               totals_out=s["totals"], blocks_out=s["blocks"])[3]
        return out, w, target, num, gone

    mine, other = state(), state()
    step(mine, inputs)                                  # the kernels and workspaces are loaded
    mine = state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(mine, inputs)
    mine["positions"].zero_()
    advanced = evicted = 0
    for i in range(60):
        inputs["qkv"].copy_(torch.randn(inputs["qkv"].shape, generator=g))
        inputs["draft"].copy_(0.3 * torch.randn(inputs["draft"].shape, generator=g))
        inputs["tokens"].copy_(torch.randint(0, V, inputs["tokens"].shape, generator=g))
        inputs["uniforms"].copy_(torch.rand(inputs["uniforms"].shape, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(other, inputs)
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
        for k in ("positions", "blocks", "totals"):
            assert torch.equal(mine[k], other[k]), (i, k)
        for k in ("block_table", "k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail"):
            assert torch.equal(getattr(mine["cache"], k), getattr(other["cache"], k)), (i, k)
        advanced += int(want[3].sum()) + B
        evicted += int(want[4].sum())
    assert int(mine["positions"].sum()) == advanced and evicted > 0
