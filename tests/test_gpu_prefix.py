"""cache_attention over prefixes that rows share, against the formula in
float64: each row as if the prefix's pages stood in its own table.

Tolerance: that of tests/test_gpu_attention.py, with 2^-8 for a probability's
rounding beside the prefix's values as beside the row's own, and what the join
of prefix and row adds: each enters with a weight from a base-2 logarithm or
exponential of at most 2 smax + 32, off by 2^-23 of that at most, so out is off
by 2 * 2^-23 (2 smax + 32) sum p |v| more, and a block's weight carries three
such logarithms instead of two.
"""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R
from tests.test_gpu_attention import make_qkv, random_parents, views

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
KINDS = ["e4m3", "int8"]


def shared_state(seed, own, shared, starts, *, Hkv, D, page, kind, spare_blocks=0, **kw):
    """(state of the rows, prefix tensors, state whose tables hold the prefixes too)."""
    B, N = len(own), len(shared)
    of = [next((i for i in range(N - 1, -1, -1) if starts[i] <= b < starts[i + 1]), None) for b in range(B)]
    before = [0 if i is None else shared[i] for i in of]
    s = R.random_state(seed, B=B + N, Hkv=Hkv, D=D, page=page, kind=kind, contexts=own + [n * page for n in shared],
                       evicted=before + [0] * N, **kw)
    most = max(shared + [1]) + spare_blocks
    table = torch.full((N, most), -1, dtype=torch.int32)
    for i in range(N):
        table[i, :shared[i]] = s["table"][B + i, :shared[i]]
    width = max([c // page for c in own] + [1]) + 1
    rows = dict(s, B=B, table=s["table"][:B, :width].contiguous(), positions=s["positions"][:B].clone(),
                blocks=s["blocks"][:B].clone(), k_tail=s["k_tail"][:B].contiguous(), v_tail=s["v_tail"][:B].contiguous())
    prefix = dict(prefix_table=table, prefix_blocks=torch.tensor(shared, dtype=torch.int32),
                  prefix_starts=torch.tensor(starts, dtype=torch.int32))
    whole = dict(rows, table=torch.full((B, most + width), -1, dtype=torch.int32),
                 blocks=rows["blocks"] + torch.tensor(before, dtype=torch.int32))
    for b in range(B):
        n = before[b]
        if n:
            whole["table"][b, :n] = table[of[b], :n]
        whole["table"][b, n:n + width] = rows["table"][b]
    return rows, prefix, whole, before


def check(whole, before, width, q, kn, vn, got, weights=None, scale=None, parents=None, query_lens=None, fill=0.0):
    D = q.shape[3]
    ref, w, av, smax = R.attention(whole, q, kn, vn, D ** -0.5 if scale is None else scale, parents, query_lens)
    rel = 2 * (D + 4) * 2.0 ** -24 * smax + 2.0 ** -20
    join = 2 * 2.0 ** -23 * (2 * smax + 32)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel + join)[..., None] * (1 + 2.0 ** -8) * av + 2.0 ** -99
    out = got.cpu().double()
    for b in range(q.shape[0]):
        n = q.shape[1] if query_lens is None else min(max(int(query_lens[b]), 0), q.shape[1])
        assert torch.isfinite(out[b, :n]).all()
        over = ((out - ref).abs() - tol)[b, :n]
        assert n == 0 or over.max() <= 0, (b, float(over.max()), float(tol[b, :n].max()))
        assert (out[b, n:] == fill).all()
        if weights is not None and n:
            x, y = weights[b, :n].cpu().double(), w[b, :n, before[b]:before[b] + width]
            r = rel[b, :n].amax(1) + 3 * 2.0 ** -23 * (2 * smax[b, :n].amax(1) + 32)
            assert ((x - y).abs() <= r[:, None] * y + 1e-30).all(), float(((x - y).abs() / y.clamp(min=1e-9)).max())
        if weights is not None:
            assert (weights[b, n:] == fill).all()


def run(rows, prefix, qkv, H, *, parents=None, query_lens=None, weights=True, **kw):
    cache, positions, blocks = R.to_gpu(rows)
    q, kn, vn = views(qkv.cuda(), H, rows["Hkv"])
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    return rsv.cache_attention(q, kn, vn, cache, positions, blocks, parents=dev(parents), query_lens=dev(query_lens),
                               weights=weights, **{k: dev(v) for k, v in prefix.items()}, **kw)


def case(seed, own, shared, starts, T, H, Hkv, D, page, kind, tree=False, query_lens=None, gain=1.0, edit=None, **kw):
    B = len(own)
    rows, prefix, whole, before = shared_state(seed, own, shared, starts, Hkv=Hkv, D=D, page=page, kind=kind, **kw)
    if edit:
        edit(rows, prefix, whole)
    qkv = make_qkv(seed + 1, B, T, H, Hkv, D, gain)
    parents = random_parents(seed + 2, B, T, bad=True) if tree else None
    if query_lens is not None:
        query_lens = torch.tensor(query_lens, dtype=torch.int32)
        for b in range(B):
            qkv[b, max(0, min(T, int(query_lens[b]))):] = float("nan")
    out, w = run(rows, prefix, qkv, H, parents=parents, query_lens=query_lens)
    width = rows["table"].shape[1]
    check(whole, before, width, *views(qkv, H, Hkv), out, w, parents=parents, query_lens=query_lens)
    plain = run(rows, prefix, qkv, H, parents=parents, query_lens=query_lens, weights=None)
    assert torch.equal(plain, out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_and_lengths(D, page, kind):
    """Prefixes of one block to several, and rows with blocks of their own, a tail alone, or nothing."""
    own = [0, 1, page - 1, page, 3 * page + 5, 7]
    case(1, own, [1, 5, 1000 // page + 1], [0, 2, 4, 6], 3, 4, 2, D, page, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H, Hkv, T", [(1, 1, 1), (8, 8, 1), (8, 1, 1), (8, 2, 2), (7, 1, 5), (6, 2, 4), (16, 2, 9),
                                       (3, 3, 33), (4, 2, 65), (200, 1, 1)])
def test_head_layouts(H, Hkv, T, kind):
    case(2, [77, 0, 30], [9], [0, 3], T, H, Hkv, 128, 32, kind)


@pytest.mark.parametrize("T", [2, 31, 61, 64])
def test_trees(T):
    case(3 + T, [0, 45, 130], [6, 3], [0, 2, 3], T, 4, 2, 64, 16, "e4m3", tree=True)


def test_rows_without_a_prefix_and_prefixes_without_rows():
    """Rows before the first group and behind the last; empty groups; a prefix of no blocks."""
    case(4, [20, 5, 40, 0, 17, 33], [4, 7, 0, 2], [1, 3, 3, 4, 5], 4, 4, 2, 64, 16, "e4m3")
    case(5, [20, 5], [3], [2, 2], 2, 4, 2, 64, 16, "int8")
    case(6, [20, 5], [3], [0, 0], 2, 4, 2, 64, 16, "int8")


def test_many_prefixes():
    """More groups than a wave looks up at once."""
    own = [5 + b % 30 for b in range(150)]
    case(7, own, [1 + i % 3 for i in range(75)], [2 * i for i in range(76)], 2, 2, 1, 64, 16, "e4m3")


@pytest.mark.parametrize("kind", KINDS)
def test_rows_beyond_a_tile_of_queries(kind):
    """Groups whose queries fill several tiles, the last one in part."""
    own = [(7 * b) % 40 for b in range(30)]
    lens = [(b * 5) % 8 - 1 for b in range(30)]
    case(8, own, [12, 5], [0, 19, 30], 6, 8, 1, 64, 16, kind, query_lens=lens)
    case(9, own, [12, 5], [0, 19, 30], 6, 8, 2, 128, 64, kind)


def test_idle_batches():
    case(10, [5, 20], [2], [0, 2], 3, 4, 2, 64, 16, "e4m3", query_lens=[0, 0])


def test_tables_far_longer_than_their_prefix():
    case(11, [5, 20, 9], [40, 1], [0, 2, 3], 3, 4, 2, 64, 16, "e4m3", spare_blocks=1000)


@pytest.mark.parametrize("gain", [0.01, 8.0, 60.0])
def test_flat_and_peaked_scores(gain):
    case(12, [50, 20, 9], [30], [0, 3], 3, 4, 2, 128, 16, "e4m3", gain=gain)


def test_pages_that_do_not_exist_are_not_seen():
    def edit(rows, prefix, whole):
        for b, (i, j) in ((0, (0, 1)), (2, (1, 0)), (2, (1, 2))):
            prefix["prefix_table"][i, j] = whole["table"][b, j] = -1 if j else 10 ** 6
        whole["table"][1, 1] = -1
    case(13, [50, 20, 9], [3, 3], [0, 2, 3], 3, 4, 2, 64, 16, "e4m3", edit=edit)

    def none(rows, prefix, whole):
        prefix["prefix_table"][:] = -1
        whole["table"][:, :3] = -1
    case(14, [50, 20], [3], [0, 2], 3, 4, 2, 64, 16, "int8", edit=none)


@pytest.mark.parametrize("kind", KINDS)
def test_value_scales_of_every_size(kind):
    """Blocks whose values are 2^-100 to 2^60 of others', at once."""
    def edit(rows, prefix, whole):
        p = prefix["prefix_table"][0]
        for j in range(8):
            rows["v_scale"][int(p[j])] *= 2.0 ** [-100, -30, -12, 0, 0, 12, 30, 60][j]
    case(15, [50, 20, 33], [8], [0, 3], 3, 4, 2, 64, 16, kind, edit=edit)


def test_nan_scales_reach_the_rows_that_see_them():
    rows, prefix, whole, before = shared_state(16, [20, 30, 40], [3, 3], [0, 2, 3], Hkv=2, D=64, page=16, kind="e4m3")
    rows["v_scale"][int(prefix["prefix_table"][0, 1]), 1] = float("nan")
    rows["k_scale"][int(prefix["prefix_table"][1, 2]), 0] = float("nan")
    qkv = make_qkv(17, 3, 2, 4, 2, 64)
    qkv[1, 0, 0] = float("nan")         # a query of head 0
    out, _ = run(rows, prefix, qkv, 4)
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[:2, :, 2:] = True
    want[2, :, :2] = True
    want[1, 0, 0] = True
    assert torch.equal(bad, want)


def test_without_a_prefix_the_bits_are_those_of_plain_attention():
    rows, prefix, _, _ = shared_state(18, [20, 300, 0], [2], [3, 3], Hkv=2, D=128, page=32, kind="e4m3")
    qkv = make_qkv(19, 3, 5, 8, 2, 128)
    out, w = run(rows, prefix, qkv, 8)
    plain, pw = run(rows, {}, qkv, 8)
    assert torch.equal(out, plain) and torch.equal(w, pw)


def test_starts_that_do_not_ascend_stay_in_bounds():
    """Starts are not checked: whatever they hold, other rows than theirs are right and nothing is written elsewhere."""
    rows, prefix, whole, before = shared_state(20, [20, 30, 40, 8], [3, 2], [0, 2, 4], Hkv=2, D=64, page=16, kind="e4m3")
    qkv = make_qkv(21, 4, 2, 4, 2, 64)
    for starts in ([5, -3, 9], [3, 1, 2], [-2 ** 31, 2 ** 31 - 1, 0]):
        prefix["prefix_starts"] = torch.tensor(starts, dtype=torch.int32)
        run(rows, prefix, qkv, 4)
    prefix["prefix_blocks"] = torch.tensor([-1, 10 ** 9], dtype=torch.int32)
    run(rows, prefix, qkv, 4)
    torch.cuda.synchronize()


def test_graphs_and_streams():
    """Replays after table, lengths and queries changed in place; calls on two streams at once."""
    B, T, H, Hkv, D, page = 6, 4, 8, 2, 64, 16
    rows, prefix, whole, before = shared_state(22, [20, 30, 40, 8, 0, 17], [9, 5], [0, 3, 6], Hkv=Hkv, D=D, page=page,
                                               kind="e4m3", spare_blocks=4)
    cache, positions, blocks = R.to_gpu(rows)
    dev = {k: v.cuda() for k, v in prefix.items()}
    qkv = make_qkv(23, B, T, H, Hkv, D).cuda()
    out = torch.zeros((B, T, H, D), dtype=BF16, device="cuda")
    w = torch.zeros((B, T, cache.max_blocks), device="cuda")

    def step(out=out, w=w, stream=None):
        q, kn, vn = views(qkv, H, Hkv)
        return rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=w, out=out, stream=stream, **dev)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        qkv.copy_(make_qkv(30 + i, B, T, H, Hkv, D))
        dev["prefix_blocks"].copy_(torch.tensor([9 - i, 1 + i]))
        dev["prefix_starts"].copy_(torch.tensor([i % 2, 2 + i, 6]))
        want, ww = step(out=None, w=True)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(w, ww)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, _ = step(out=None, w=True, stream=side.cuda_stream)
    b, _ = step(out=None, w=True)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_refusals_on_device_tensors():
    rows, prefix, _, _ = shared_state(24, [20, 30], [3, 2], [0, 1, 2], Hkv=2, D=64, page=16, kind="e4m3")
    qkv = make_qkv(25, 2, 2, 4, 2, 64)

    def refused(err=ValueError, **kw):
        with pytest.raises(err):
            run(rows, {k: v for k, v in dict(prefix, **kw).items() if v is not None}, qkv, 4)
    refused(prefix_table=None)
    refused(prefix_blocks=None)
    refused(prefix_starts=None)
    refused(prefix_table=prefix["prefix_table"].long())
    refused(prefix_table=prefix["prefix_table"][0])
    refused(prefix_table=prefix["prefix_table"][:, :0])
    refused(prefix_blocks=prefix["prefix_blocks"][:1])
    refused(prefix_starts=prefix["prefix_starts"][:2])
    with pytest.raises(rsv.SpecVerifyError):
        run(rows, prefix, qkv, 4, workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
