"""cache_attention against the formula in float64, on the GPU.

Tolerance.  A score is a float32 sum of D exact products (bf16 times a code,
or bf16 times bf16) times the block's scale and the softmax scale: off by at
most (D + 4) 2^-24 times the sum of the products' magnitudes, smax at most,
so a probability is off by 2 (D + 4) 2^-24 smax relative (itself and the
denominator), plus 2^-20 for the exponentials (of arguments below 2^4 after
the maximum where they matter), the sums over a lane's keys and the joins.
Call this rel.  A probability times its scale is rounded to bf16 (2^-8), the
output sum is float32, and the output is rounded to bf16 (2^-8):
  |out - ref| <= 2^-8 |ref| + (2^-8 + rel) (1 + 2^-8) sum p |v| + 2^-99
the last term for float32's range: an exponential below 2^-126 may be lost
whole, and at most 2^15 keys with values below 2^11 times 2^-126 make 2^-100
(rounding a bf16 below its normal range, 2^-126, is off by less still).
A block's weight carries rel and the rounding of two base-2 logarithms of
at most 2 smax + 32 each, 2^-23 of that at most.
"""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def make_qkv(seed, B, T, H, Hkv, D, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g)
    qkv[:, :, :H] *= gain
    return qkv.to(BF16)


def views(qkv, H, Hkv):
    return qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]


def random_parents(seed, B, T, bad=False):
    g = torch.Generator().manual_seed(seed)
    par = torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        for c in range(1, T):
            par[b, c] = torch.randint(max(0, c - 4), c, (1,), generator=g)
        if bad and T > 3:
            par[b, 2], par[b, 3] = 2, -5
    return par


def check(s, q, kn, vn, got, weights=None, scale=None, parents=None, query_lens=None, fill=0.0):
    D = q.shape[3]
    ref, w, av, smax = R.attention(s, q, kn, vn, D ** -0.5 if scale is None else scale, parents, query_lens)
    rel = 2 * (D + 4) * 2.0 ** -24 * smax + 2.0 ** -20
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel[..., None]) * (1 + 2.0 ** -8) * av + 2.0 ** -99
    out = got.cpu().double()
    for b in range(q.shape[0]):
        n = q.shape[1] if query_lens is None else min(max(int(query_lens[b]), 0), q.shape[1])
        assert torch.isfinite(out[b, :n]).all()
        over = ((out - ref).abs() - tol)[b, :n]
        assert n == 0 or over.max() <= 0, (b, float(over.max()))
        assert (out[b, n:] == fill).all()
        if weights is not None and n:
            x, y = weights[b, :n].cpu().double(), w[b, :n]
            r = rel[b, :n].amax(1) + 2 * 2.0 ** -23 * (2 * smax[b, :n].amax(1) + 32)
            assert ((x - y).abs() <= r[:, None] * y + 1e-30).all(), float(((x - y).abs() / y.clamp(min=1e-9)).max())
        if weights is not None:
            assert (weights[b, n:] == fill).all()


def run(s, qkv, H, *, parents=None, query_lens=None, scale=None, weights=True, **kw):
    cache, positions, blocks = R.to_gpu(s)
    q, kn, vn = views(qkv.cuda(), H, s["Hkv"])
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    return rsv.cache_attention(q, kn, vn, cache, positions, blocks, parents=dev(parents), query_lens=dev(query_lens),
                               scale=scale, weights=weights, **kw)


def case(seed, contexts, T, H, Hkv, D, page, kind, tree=False, query_lens=None, gain=1.0, **kw):
    B = len(contexts)
    s = R.random_state(seed, B=B, Hkv=Hkv, D=D, page=page, kind=kind, contexts=contexts, **kw)
    qkv = make_qkv(seed + 1, B, T, H, Hkv, D, gain)
    parents = random_parents(seed + 2, B, T, bad=True) if tree else None
    if query_lens is not None:
        query_lens = torch.tensor(query_lens, dtype=torch.int32)
        for b in range(B):
            qkv[b, max(0, min(T, int(query_lens[b]))):] = float("nan")
    out, w = run(s, qkv, H, parents=parents, query_lens=query_lens)
    check(s, *views(qkv, H, Hkv), out, w, parents=parents, query_lens=query_lens)
    plain = run(s, qkv, H, parents=parents, query_lens=query_lens, weights=None)
    assert torch.equal(plain, out)


KINDS = ["e4m3", "int8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_and_lengths(D, page, kind):
    case(1, [0, 1, page - 1, page, page + 1, 3 * page + 5, 7 * page, 1000], 3, 4, 2, D, page, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H, Hkv, T", [(1, 1, 1), (8, 8, 1), (8, 1, 1), (8, 2, 2), (7, 1, 5), (6, 2, 4), (16, 1, 2),
                                       (16, 2, 9), (3, 3, 33), (4, 2, 65)])
def test_head_layouts(H, Hkv, T, kind):
    case(2, [77, 0, 300], T, H, Hkv, 128, 32, kind)


@pytest.mark.parametrize("D, page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("T", [1, 2, 5, 31, 32, 33, 61, 64])
def test_trees_with_bad_parents(T, D, page):
    case(3 + T, [0, 45, 130], T, 4, 2, D, page, "e4m3", tree=True)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_rows_with_fewer_tokens_and_idle_rows(page, tree):
    case(4, [200, 33, 0, 64, 5, 400], 9, 4, 2, 64, page, "e4m3", tree=tree, query_lens=[9, 0, 1, 5, -3, 12])


@pytest.mark.parametrize("kind", KINDS)
def test_evicted_rows_and_wrapped_rings(kind):
    case(5, [100, 31, 64, 200], 4, 4, 1, 64, 32, kind, evicted=[7, 1, 1000, 3])


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_missing_pages_are_not_seen(page, kind):
    """Their clamped stand-in holds NaN codes or scales, none of which may leak."""
    n = 6
    case(6, [n * page + 3, n * page], 3, 4, 2, 64, page, kind,
         bad_entries=[(0, 0, -1), (0, 3, 2 ** 31 - 1), (1, 5, -2 ** 31), (1, 1, 10 ** 6), (1, 2, -1)])


@pytest.mark.parametrize("kind", KINDS)
def test_long_contexts_are_split_and_joined(kind):
    case(7, [20011, 3, 5000], 2, 4, 1, 64, 64, kind)


def test_many_rows_of_ragged_lengths():
    case(8, [(37 * b) % 150 for b in range(300)], 2, 2, 1, 64, 16, "e4m3")


def test_scores_of_every_size():
    """Large queries: one key takes all, the others' exponentials vanish."""
    case(9, [500, 70], 3, 4, 2, 64, 64, "e4m3", gain=40.0)
    case(10, [500, 70], 3, 4, 2, 64, 16, "int8", gain=0.001)


def test_every_code_is_its_value():
    """One key per block takes all of the softmax; its value, each code in turn, comes back."""
    for kind in KINDS:
        D, page = 64, 16
        codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
        s = R.random_state(11, B=4, Hkv=1, D=D, page=page, kind=kind, contexts=[page] * 4)
        for b in range(4):
            p = int(s["table"][b, 0])
            s["k_pages"][p] = 0
            s["k_pages"][p, 0, 5] = 0x38 if kind == "e4m3" else 1  # 1.0
            v = codes[b * D:(b + 1) * D].clone()
            if kind == "e4m3":
                v = torch.where((v & 0x7F) == 0x7F, 0, v)
            s["v_pages"][p] = 0
            s["v_pages"][p, 0, :, 5] = v
            s["k_scale"][p], s["v_scale"][p] = 1.0, 1.0
        qkv = torch.zeros((4, 1, 3, D))
        qkv[:, :, 0] = 16.0
        qkv[:, :, 1] = -16.0
        out = run(s, qkv.to(BF16), 1, weights=None)
        for b in range(4):
            want = R.decode(s["v_pages"][int(s["table"][b, 0]), 0, :, 5], kind)
            assert torch.equal(out[b, 0, 0].cpu().double(), want), (kind, b)


@pytest.mark.parametrize("H, Hkv, D, T", [(4, 2, 64, 12), (8, 2, 128, 40), (32, 2, 64, 9), (2, 2, 128, 5)])
@pytest.mark.parametrize("tree", [False, True])
def test_infinities_and_nan_reach_only_the_queries_that_see_them(tree, H, Hkv, D, T):
    contexts = [40, 0, 130, 700]
    s = R.random_state(31, B=4, Hkv=Hkv, D=D, page=32, kind="e4m3", contexts=contexts)
    qkv = make_qkv(32, 4, T, H, Hkv, D)
    parents = random_parents(33, 4, T) if tree else None
    v = qkv[:, :, H + Hkv:]
    v[:, 2, 0, 3], v[:, 2, 0, D - 1], v[:, 2, 0, 17] = float("inf"), float("-inf"), float("nan")
    v[:, T - 1, 1, :] = float("nan")
    v[0, 1, 1, 8:12] = float("inf")
    qkv[:, 4, H + 1, 5] = float("nan")                      # a key of the second head
    s["v_tail"][2, int(R.tail_slots(s, 2, s["v_tail"].shape[1])[0]), 0, 9] = float("inf")
    q, kn, vn = views(qkv, H, Hkv)
    got = run(s, qkv, H, parents=parents, weights=None).cpu().double()
    ref, _, av, smax = R.attention(s, q, kn, vn, D ** -0.5, parents)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert not torch.isinf(got[~torch.isinf(ref)]).any()
    fine = torch.isfinite(ref)
    assert fine[:, 0].sum() > H * D and not fine.all()
    rel = 2 * (D + 4) * 2.0 ** -24 * smax + 2.0 ** -20
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel[..., None]) * (1 + 2.0 ** -8) * av + 2.0 ** -99
    assert ((got - ref).abs() <= tol)[fine].all()


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_nan_scales_reach_every_query_that_sees_the_block(which):
    s = R.random_state(12, B=2, Hkv=2, D=64, page=16, kind="e4m3", contexts=[100, 100])
    s[which][int(s["table"][1, 2]), 1] = float("nan")
    qkv = make_qkv(13, 2, 2, 4, 2, 64)
    out = run(s, qkv, 4, weights=None).float()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :, :2]).all()
    assert torch.isnan(out[1, :, 2:]).all()


def test_offsets_past_32_bits():
    Hkv, D, page = 8, 128, 64
    pages = 2 ** 32 // (Hkv * D * page) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * pages * Hkv * D * page:
        pytest.skip("too little memory")
    s = R.random_state(14, B=2, Hkv=Hkv, D=D, page=page, kind="e4m3", contexts=[5 * page + 9, 3 * page])
    qkv = make_qkv(15, 2, 3, 16, Hkv, D)
    want, ww = run(s, qkv, 16)
    cache, positions, blocks = R.to_gpu(s)
    small = s["k_pages"].shape[0]
    shift = pages - small
    big = {}
    for k in ("k_pages", "v_pages", "k_scale", "v_scale"):
        t = getattr(cache, k)
        big[k] = torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
        big[k][shift:] = t
    table = torch.where(cache.block_table >= 0, cache.block_table + shift, -1)
    far = rsv.KVCache(big["k_pages"], big["v_pages"], big["k_scale"], big["v_scale"], cache.k_tail, cache.v_tail, table)
    q, kn, vn = views(qkv.cuda(), 16, Hkv)
    out, w = rsv.cache_attention(q, kn, vn, far, positions, blocks, weights=True)
    assert torch.equal(out, want) and torch.equal(w, ww)


def test_results_are_reproducible_and_rows_independent():
    contexts = [900, 64, 0, 333, 2000]
    s = R.random_state(16, B=5, Hkv=2, D=128, page=64, kind="e4m3", contexts=contexts)
    qkv = make_qkv(17, 5, 6, 8, 2, 128)
    a, wa = run(s, qkv, 8)
    b, wb = run(s, qkv, 8)
    assert torch.equal(a, b) and torch.equal(wa, wb)


def test_given_outputs_workspace_and_streams():
    s = R.random_state(18, B=3, Hkv=2, D=64, page=16, kind="int8", contexts=[300, 17, 40])
    qkv = make_qkv(19, 3, 5, 4, 2, 64)
    ql = torch.tensor([5, 2, 0], dtype=torch.int32)
    cache, positions, blocks = R.to_gpu(s)
    q, kn, vn = views(qkv.cuda(), 4, 2)
    out = torch.full((3, 5, 4, 64), 7.0, dtype=BF16, device="cuda")
    w = torch.full((3, 5, cache.max_blocks), 7.0, device="cuda")
    ws = rsv.new_attention_workspace(cache, 5, 4, weights=True)
    assert ws.numel() == rsv.attention_workspace_bytes(cache, 5, 4, weights=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = rsv.cache_attention(q, kn, vn, cache, positions, blocks, query_lens=ql.cuda(), out=out, weights=w,
                              workspace=ws, stream=side.cuda_stream)
    side.synchronize()
    assert got[0] is out and got[1] is w
    check(s, *views(qkv, 4, 2), out, w, query_lens=ql, fill=7.0)


def test_a_workspace_serves_calls_of_its_shape_one_after_the_other():
    """Lengths and idle rows change between calls; the counters come back to zero whatever the last call was."""
    B, T, H, Hkv, D, page = 4, 3, 4, 1, 64, 64
    ws = None
    for i, (contexts, lens) in enumerate([([9000, 10, 0, 4000], None), ([100, 8000, 5000, 1], [3, 0, 2, 3]),
                                          ([9999, 0, 9999, 77], [0, 0, 1, 3]), ([9000, 10, 0, 4000], None)]):
        s = R.random_state(60 + i, B=B, Hkv=Hkv, D=D, page=page, kind="e4m3", contexts=contexts, max_blocks=160)
        qkv = make_qkv(70 + i, B, T, H, Hkv, D)
        lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
        cache, _, _ = R.to_gpu(s)
        ws = rsv.new_attention_workspace(cache, T, H, weights=True) if ws is None else ws
        out, w = run(s, qkv, H, query_lens=lens, workspace=ws)
        check(s, *views(qkv, H, Hkv), out, w, query_lens=lens)
        assert not ws[:B * Hkv * 4].any()


def test_many_query_heads_per_kv_head():
    case(80, [70, 0, 5], 3, 256, 1, 64, 16, "e4m3")
    case(81, [70, 200], 2, 400, 2, 128, 64, "int8", query_lens=[2, 1])


def test_more_rows_than_a_wave_and_trees_of_all_sizes():
    contexts = [(53 * b) % 300 for b in range(70)]
    case(82, contexts, 33, 4, 2, 64, 16, "e4m3", tree=True, query_lens=[(7 * b) % 34 for b in range(70)])


def test_graph_replays_follow_the_lengths():
    B, H, Hkv, D, page, T = 3, 4, 2, 64, 16, 4
    states = [R.random_state(20 + i, B=B, Hkv=Hkv, D=D, page=page, kind="e4m3", contexts=c, max_blocks=130,
                             spare=200 - sum(x // page for x in c))
              for i, c in enumerate([[5, 100, 40], [2000, 0, 16], [33, 650, 64]])]
    cache, positions, blocks = R.to_gpu(states[0])
    qkv = make_qkv(30, B, T, H, Hkv, D).cuda()
    q, kn, vn = views(qkv, H, Hkv)
    out, w = rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rsv.cache_attention(q, kn, vn, cache, positions, blocks, out=out, weights=w)
    for i in (1, 2, 0, 1, 1):
        s = states[i]
        for k in R.TENSORS:
            getattr(cache, "block_table" if k == "table" else k).copy_(s[k])
        positions.copy_(s["positions"])
        blocks.copy_(s["blocks"])
        qkv.copy_(make_qkv(40 + i, B, T, H, Hkv, D))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(s, *views(qkv.cpu(), H, Hkv), out, w)
        eager = rsv.cache_attention(q, kn, vn, cache, positions, blocks, weights=True)
        assert torch.equal(out, eager[0]) and torch.equal(w, eager[1])


def test_outputs_between_the_rows_that_are_read():
    """One allocation: q's rows apart, the output in the gap between two of them; over a row it is refused."""
    B, T, H, Hkv, D = 3, 2, 4, 2, 64
    s = R.random_state(60, B=B, Hkv=Hkv, D=D, page=16, kind="int8", contexts=[20, 0, 300])
    qkv = make_qkv(61, B, T, H, Hkv, D)
    cache, positions, blocks = R.to_gpu(s)
    _, kn, vn = views(qkv.cuda(), H, Hkv)
    n, size = T * H * D, B * T * H * D
    arena = torch.zeros((B * (n + size),), dtype=BF16, device="cuda")
    q = arena.as_strided((B, T, H, D), (n + size, H * D, D, 1))
    q.copy_(qkv[:, :, :H])
    for row in range(B):
        out = arena[row * (n + size) + n:][:size].view(B, T, H, D)
        rsv.cache_attention(q, kn, vn, cache, positions, blocks, out=out)
        check(s, *views(qkv, H, Hkv), out)
        for at in (row * (n + size) + n - 8, (row + 1) * (n + size) - size + 8):
            if row < B - 1 or at < row * (n + size) + n:
                with pytest.raises(rsv.SpecVerifyError):
                    rsv.cache_attention(q, kn, vn, cache, positions, blocks, out=arena[at:at + size].view(B, T, H, D))
    with pytest.raises(rsv.SpecVerifyError):
        rsv.cache_attention(q, kn, vn, cache, positions, blocks, out=arena[8:8 + size].view(B, T, H, D))


def test_a_cache_keeps_its_tensors():
    s = R.random_state(62, B=1, Hkv=1, D=64, page=16, kind="int8", contexts=[20])
    cache, _, _ = R.to_gpu(s)
    with pytest.raises(AttributeError):
        cache.block_table = cache.block_table.clone()
    with pytest.raises(AttributeError):
        cache.page = 32


def test_refusals_on_device_tensors():
    s = R.random_state(50, B=2, Hkv=2, D=64, page=16, kind="e4m3", contexts=[20, 40])
    cache, positions, blocks = R.to_gpu(s)
    q, kn, vn = views(make_qkv(51, 2, 3, 4, 2, 64).cuda(), 4, 2)
    def refused(err=ValueError, q=q, kn=kn, vn=vn, cache=cache, positions=positions, blocks=blocks, **kw):  # noqa: E306
        with pytest.raises(err):
            rsv.cache_attention(q, kn, vn, cache, positions, blocks, **kw)
    refused(q=q.float())
    refused(q=q.transpose(1, 2))
    refused(q=q[:, :, :, :32])
    refused(q=q[:1])
    refused(kn=kn[:, :2])
    refused(kn=kn.contiguous())                      # other strides than v_new
    refused(cache=None)
    refused(positions=positions.long())
    refused(blocks=blocks[:1])
    refused(parents=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))
    refused(query_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    refused(out=torch.zeros((2, 3, 4, 64), device="cuda"))
    refused(weights=torch.zeros((2, 3, 1), device="cuda"))
    refused(rsv.SpecVerifyError, scale=0.0)
    refused(rsv.SpecVerifyError, scale=float("nan"))
    refused(rsv.SpecVerifyError, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros((2, 3, 8 * 64 + 4), dtype=BF16, device="cuda")
    refused(q=wide[:, :, 4:].unflatten(2, (8, 64))[:, :, :4])  # 8-byte aligned
    t = R.TENSORS
    parts = {k: getattr(cache, "block_table" if k == "table" else k) for k in t}
    for k, v in (("k_pages", parts["k_pages"].view(torch.int8)), ("v_pages", parts["k_pages"]), ("k_scale", None),
                 ("v_tail", parts["v_tail"][:1]), ("table", parts["table"].long())):
        with pytest.raises(ValueError):
            rsv.KVCache(*(dict(parts, **{k: v})[x] for x in t))
    with pytest.raises(ValueError):
        rsv.KVCache(*(parts[x] for x in t), kind="fp8")
