"""cache_append against its definition, on the GPU: the cache that it leaves is
compared, to the bit, with the reference of a commit of the rotated keys, and
with what rotate_tokens and cache_commit leave."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R
from tests import rotary_ref as RR
from tests.test_gpu_commit import check, random_new, state_with_reserve
from tests.test_gpu_rotate import freqs_of, near

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
KINDS = ["e4m3", "int8"]


def case(seed, contexts, lens, T, Hkv, D, page, kind, dims=None, interleaved=False, ids=None, axes=None, max_new=65,
         edit=None, evicted=None, spread=1.0):
    """dims: rotated channels (None: all, 0: no rotation)."""
    B = len(contexts)
    reserve = -(-(page - 1 + T) // page)
    s = state_with_reserve(seed, reserve, B=B, Hkv=Hkv, D=D, page=page, kind=kind, contexts=contexts, max_new=max_new,
                           evicted=evicted)
    kv = random_new(seed + 1, B, T, Hkv, D, spread)
    if edit:
        edit(s, kv)
    dims = D if dims is None else dims
    n = torch.full((B,), T, dtype=torch.int32) if lens is None else torch.tensor(lens, dtype=torch.int32)
    freqs = freqs_of(dims) if dims else None
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache, positions, blocks = R.to_gpu(s)
    kvd = kv.cuda()
    rot = dict(freqs=dev(freqs), interleaved=interleaved, ids=dev(ids), axes=dev(axes))
    k_out = torch.zeros((B, T, Hkv, D), dtype=BF16, device="cuda")
    outs = rsv.cache_append(cache, kvd[:, :, 0], kvd[:, :, 1], positions, blocks, lens=None if lens is None else dev(n),
                            k_out=k_out, **rot)
    assert torch.equal(kvd.cpu().view(torch.int16), kv.view(torch.int16))
    rotated = kv.clone()
    if dims:
        turned, _ = rsv.rotate_tokens(kvd[:, :, 0], kvd[:, :, 0], freqs.cuda(), positions, interleaved=interleaved,
                                      ids=dev(ids), axes=dev(axes))
        rotated[:, :, 0] = turned.cpu()
        at = RR.token_positions(s["positions"], T)[None] if ids is None else ids
        sound = [0 <= int(n[b]) <= T for b in range(B)]
        near(turned, kv[:, :, 0], freqs, interleaved, at, axes)
        assert all(sound) or edit
    want = check(s, rotated, n - 1, cache, outs)
    for b in range(B):
        done = int(want["positions"][b] - s["positions"][b])
        assert torch.equal(k_out[b, :done].cpu().view(torch.int16), rotated[b, :done, 0].view(torch.int16))
        assert (k_out[b, done:] == 0).all()
    # in place: counters, and the rotated keys over the keys
    cache2, pos2, blk2 = R.to_gpu(s)
    res = rsv.cache_append(cache2, kvd[:, :, 0], kvd[:, :, 1], pos2, blk2, lens=dev(n), k_out=kvd[:, :, 0],
                           positions_out=pos2, blocks_out=blk2, **rot)
    check(s, rotated, n - 1, cache2, res)
    assert res[0] is pos2 and res[1] is blk2
    for b in range(B):
        done = int(want["positions"][b] - s["positions"][b])
        assert torch.equal(kvd[b, :done, 0].view(torch.int16), k_out[b, :done].view(torch.int16))
        assert torch.equal(kvd[b, done:].cpu().view(torch.int16), kv[b, done:].view(torch.int16))
    assert torch.equal(kvd[:, :, 1].cpu().view(torch.int16), kv[:, :, 1].view(torch.int16))
    return want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_and_lengths(D, page, kind):
    contexts = [0, 1, page - 1, page, 2 * page + page // 2, page - 3]
    lens = [3 * page, 0, 1, page - 1, page, 2 * page + 5]
    case(1, contexts, lens, 3 * page, 2, D, page, kind)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [0, 16, 64, 128])
def test_rotated_channels(dims, interleaved):
    case(2, [5, 100], [130, 67], 130, 3, 128, 64, "e4m3", dims=dims, interleaved=interleaved)
    case(3, [5, 300], [300, 257], 300, 1, 128, 256, "int8", dims=dims, interleaved=interleaved)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 1000])
def test_lengths(T):
    case(4, [0, 63, 17], None, T, 2, 64, 64, "e4m3")


def test_positions_of_three_axes():
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, 100000, (3, 2, 90), generator=g, dtype=torch.int32)
    axes = torch.randint(0, 3, (32,), generator=g, dtype=torch.int32)
    case(5, [3, 40], [90, 71], 90, 2, 64, 32, "e4m3", ids=ids, axes=axes)


@pytest.mark.parametrize("kind", KINDS)
def test_rings_of_one_block(kind):
    """The new tail lies where the old one was, which is read first."""
    case(6, [15, 7, 31, 8], [17, 40, 33, 16], 40, 2, 64, 16, kind, max_new=1)


def test_far_evicted_rows():
    case(7, [47, 31], [30, 64], 64, 2, 64, 16, "e4m3", evicted=[100, 100000])


@pytest.mark.parametrize("kind", KINDS)
def test_values_of_every_size(kind):
    def edit(s, kv):
        kv[0] = 0
        s["k_tail"][0] = 0
        s["v_tail"][0] = 0
        kv[1] *= 2.0 ** -120
        kv[2] *= 2.0 ** 100
    case(8, [15, 16, 16, 10], None, 16, 2, 64, 16, kind, spread=3.0, edit=edit)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_blocks_with_infinities_or_nan_get_a_nan_scale(bad):
    def edit(s, kv):
        kv[0, 2, 0, 1, 5] = bad
        kv[1, 20, 1, 0, 63] = bad
    case(9, [15, 12], None, 40, 2, 64, 16, "e4m3", dims=0, edit=edit)


def test_rows_left_as_they_were():
    """Impossible lengths and counters; rows without a page for the first or for the last block that they complete."""
    def edit(s, kv):
        s["table"][3, int(s["blocks"][3])] = -1
        s["table"][4, int(s["blocks"][4]) + 2] = 10 ** 6
        s["positions"][5] = -5
        s["blocks"][6] = 100
        s["blocks"][7] = -1
        s["positions"][8] = 2 ** 31 - 3
        s["blocks"][9] = s["table"].shape[1] - 1
    want = case(10, [15] * 11, [-1, 51, 0, 40, 40, 3, 3, 3, 5, 50, 40], 50, 2, 64, 16, "e4m3", edit=edit, dims=0)
    assert want["positions"].tolist()[:4] == [15, 15, 15, 15] and int(want["positions"][10]) == 55


def test_equals_chains_of_commits():
    """A prompt in one call, and as chains of up to 65 tokens: the same cache."""
    B, T, Hkv, D, page = 2, 150, 2, 64, 32
    s = state_with_reserve(11, 6, B=B, Hkv=Hkv, D=D, page=page, kind="int8", contexts=[3, 40])
    kv = random_new(12, B, T, Hkv, D).cuda()
    freqs = freqs_of(D).cuda()
    cache, positions, blocks = R.to_gpu(s)
    got = rsv.cache_append(cache, kv[:, :, 0], kv[:, :, 1], positions, blocks, freqs=freqs)
    other, positions, blocks = R.to_gpu(s)
    for t in range(0, T, 65):
        part = kv[:, t:t + 65]
        n = part.shape[1]
        k, _ = rsv.rotate_tokens(part[:, :, 0], part[:, :, 0], freqs, positions)
        v = part[:, :, 1].contiguous()
        accepted = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
        positions, blocks = rsv.cache_commit(other, k, v, accepted, positions, blocks)
    assert torch.equal(got[0], positions) and torch.equal(got[1], blocks)
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, name).view(torch.uint8), getattr(other, name).view(torch.uint8)), name
    for b in range(B):
        new = dict(s, positions=positions.cpu())
        for slot in R.tail_slots(new, b, cache.tail):
            for x in ("k_tail", "v_tail"):
                assert torch.equal(getattr(cache, x)[b, slot], getattr(other, x)[b, slot])


def test_many_rows_share_work_groups_between_heads():
    """Enough blocks that a work-group takes several heads."""
    B, T = 48, 64 * 45
    s = state_with_reserve(13, 46, B=B, Hkv=3, D=64, page=64, kind="e4m3", contexts=[b % 64 for b in range(B)])
    kv = random_new(14, 1, T, 3, 64).expand(B, T, 2, 3, 64).contiguous()
    cache, positions, blocks = R.to_gpu(s)
    kvd = kv.cuda()
    n = torch.tensor([T - 37 * b for b in range(B)], dtype=torch.int32)
    outs = rsv.cache_append(cache, kvd[:, :, 0], kvd[:, :, 1], positions, blocks, lens=n.cuda())
    check(s, kv, n - 1, cache, outs)


def test_graph_replays_advance_in_place():
    B, T, Hkv, D, page = 2, 40, 2, 64, 16
    s = state_with_reserve(15, 12, B=B, Hkv=Hkv, D=D, page=page, kind="e4m3", contexts=[3, 30])
    cache, positions, blocks = R.to_gpu(s)
    kv = random_new(16, B, T, Hkv, D).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    step = lambda: rsv.cache_append(cache, kv[:, :, 0], kv[:, :, 1], positions, blocks, lens=lens,  # noqa: E731
                                    positions_out=positions, blocks_out=blocks)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        kv.copy_(random_new(20 + i, B, T, Hkv, D))
        lens.copy_(torch.tensor([10 * i + 1, 40]))
        before = dict(s, **{k: getattr(cache, "block_table" if k == "table" else k).cpu() for k in R.TENSORS},
                      positions=positions.cpu(), blocks=blocks.cpu())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(before, kv.cpu(), lens.cpu() - 1, cache, (positions, blocks))


def test_refusals_on_device_tensors():
    s = state_with_reserve(17, 2, B=2, Hkv=2, D=64, page=16, kind="e4m3", contexts=[5, 15])
    cache, positions, blocks = R.to_gpu(s)
    kv = random_new(18, 2, 3, 2, 64).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")

    def refused(err=ValueError, k=kv[:, :, 0], v=kv[:, :, 1], positions=positions, blocks=blocks, **kw):
        with pytest.raises(err):
            rsv.cache_append(cache, k, v, positions, blocks, **kw)
    refused(k=kv[:, :, 0].float())
    refused(v=kv[:, :, 1].contiguous())
    refused(positions=positions.long())
    refused(lens=torch.zeros(3, **i32))
    refused(ids=torch.zeros((1, 2, 3), **i32))                       # no freqs
    refused(freqs=torch.zeros(33, device="cuda"))
    refused(k_out=kv[:, :, 0].float())
    refused(rsv.SpecVerifyError, freqs=torch.zeros(4, device="cuda"))
    refused(rsv.SpecVerifyError, k_out=kv[:, :, 1])                  # over the values
    refused(rsv.SpecVerifyError, positions_out=positions)            # one counter in place alone
    refused(rsv.SpecVerifyError, k_out=cache.k_tail[:, :3])
