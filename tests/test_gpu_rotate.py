"""rotate_tokens against the rotation in 64 bits (the bound is derived in
tests/rotary_ref.py), on the GPU."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import rotary_ref as RR

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def freqs_of(dims, base=10000.0):
    return (base ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)).float()


def tree(seed, B, T):
    g = torch.Generator().manual_seed(seed)
    par = torch.zeros((B, T), dtype=torch.int32)
    for t in range(1, T):
        par[:, t] = torch.randint(max(0, t - 5), t, (B,), generator=g).to(torch.int32)
    return par


def inputs(seed, B, T, H, Hkv, D):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g) * torch.exp(2 * torch.randn((B, T, 1, 1), generator=g))
    return qkv.to(BF16)


def near(got, x, freqs, interleaved, ids, axes, lens=None):
    y, off = RR.rotate(x, freqs, interleaved, ids, axes)
    got = got.cpu().double()
    for b in range(x.shape[0]):
        n = x.shape[1] if lens is None else min(max(int(lens[b]), 0), x.shape[1])
        assert ((got[b, :n] - y[b, :n]).abs() <= off[b, :n]).all(), float(((got - y).abs() / off)[b, :n].max())
        assert (got[b, n:] == 0).all()
    dims = 2 * freqs.shape[0]
    live = got[..., dims:] == x[..., dims:].double()
    assert live.all() or lens is not None


def case(seed, B, T, H, Hkv, D, dims, positions, interleaved=False, parents=None, lens=None, ids=None, axes=None):
    qkv = inputs(seed, B, T, H, Hkv, D)
    freqs = freqs_of(dims)
    positions = torch.tensor(positions, dtype=torch.int32)
    at = RR.token_positions(positions, T, parents)[None] if ids is None else ids
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    x = qkv.cuda()
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    kw = dict(interleaved=interleaved, parents=dev(parents), query_lens=dev(lens), ids=dev(ids), axes=dev(axes))
    q, k = rsv.rotate_tokens(x[:, :, :H], x[:, :, H:H + Hkv], freqs.cuda(), positions.cuda(), **kw)
    near(q, qkv[:, :, :H], freqs, interleaved, at, axes, lens)
    near(k, qkv[:, :, H:H + Hkv], freqs, interleaved, at, axes, lens)
    assert torch.equal(x.cpu().view(torch.int16), qkv.view(torch.int16))
    # in place, inside the projection's output: the same bits, the values and what lies behind the lengths untouched
    rsv.rotate_tokens(x[:, :, :H], x[:, :, H:H + Hkv], freqs.cuda(), positions.cuda(), q_out=x[:, :, :H],
                      k_out=x[:, :, H:H + Hkv], **kw)
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        assert torch.equal(x[b, :n, :H], q[b, :n]) and torch.equal(x[b, :n, H:H + Hkv], k[b, :n])
        assert torch.equal(x[b, n:].cpu(), qkv[b, n:])
    assert torch.equal(x[:, :, H + Hkv:].cpu(), qkv[:, :, H + Hkv:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D, dims", [(64, 64), (128, 128), (128, 64), (128, 16), (80, 80), (96, 32), (256, 256), (512, 512),
                                     (16, 16)])
def test_channels(D, dims, interleaved):
    case(1, 3, 5, 6, 2, D, dims, [0, 77, 4095], interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles of up to 2^31 radians: their turns are counted in 64 bits."""
    case(2, 6, 3, 2, 1, 128, 128, [2 ** 17, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 30, 2 ** 31 - 4, 2 ** 31 - 1], interleaved)


@pytest.mark.parametrize("T", [2, 17, 61, 64])
def test_trees(T):
    par = tree(T, 3, T)
    par[1, T // 2] = T          # paths that start at a node whose parent is not an earlier one
    par[2, 1] = -1
    case(3, 3, T, 4, 2, 64, 64, [5, 1000, 131072], parents=par)


def test_chain_as_a_tree():
    par = torch.arange(-1, 63, dtype=torch.int32)[None].contiguous()
    case(4, 1, 64, 4, 1, 64, 64, [9], parents=par)


@pytest.mark.parametrize("B, T", [(1, 1), (4, 65), (2, 3000), (5000, 1)])
def test_lengths_and_rows(B, T):
    """Both forms of the kernel: one token to a work-group, and four."""
    case(5, B, T, 3, 1, 64, 32, [7 * b for b in range(B)], lens=[(3 * b) % (T + 2) - 1 for b in range(B)] if T > 1 else None)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_three_axes(interleaved):
    g = torch.Generator().manual_seed(6)
    ids = torch.randint(-50, 200000, (3, 2, 9), generator=g, dtype=torch.int32)
    axes = torch.randint(-1, 5, (32,), generator=g, dtype=torch.int32)   # taken into [0, 3)
    case(6, 2, 9, 4, 2, 64, 64, [0, 0], interleaved, ids=ids, axes=axes, lens=[9, 4])
    case(7, 2, 9, 4, 2, 64, 64, [0, 0], interleaved, ids=ids)


def test_infinities_stay_in_their_pair():
    x = torch.ones((1, 2, 2, 64), dtype=BF16)
    x[0, 0, 0, 3] = float("inf")
    x[0, 1, 1, 40] = float("nan")
    q, k = rsv.rotate_tokens(x.cuda(), x.cuda(), freqs_of(64).cuda(), torch.tensor([5], dtype=torch.int32).cuda())
    bad = ~torch.isfinite(q.cpu())
    want = torch.zeros_like(bad)
    want[0, 0, 0, [3, 35]] = True
    want[0, 1, 1, [8, 40]] = True
    assert torch.equal(bad, want) and torch.equal(~torch.isfinite(k.cpu()), want)


def test_graph_and_streams():
    B, T, H, Hkv, D = 4, 6, 8, 2, 128
    qkv = inputs(8, B, T, H, Hkv, D).cuda()
    freqs, pos = freqs_of(D).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = (torch.zeros((B, T, H, D), dtype=BF16, device="cuda"), torch.zeros((B, T, Hkv, D), dtype=BF16, device="cuda"))
    step = lambda: rsv.rotate_tokens(qkv[:, :, :H], qkv[:, :, H:H + Hkv], freqs, pos, q_out=outs[0], k_out=outs[1])  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        qkv.copy_(inputs(20 + i, B, T, H, Hkv, D))
        pos.add_(1000 * i + 7)
        want = rsv.rotate_tokens(qkv[:, :, :H], qkv[:, :, H:H + Hkv], freqs, pos)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rsv.rotate_tokens(qkv[:, :, :H], qkv[:, :, H:H + Hkv], freqs, pos, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_on_device_tensors():
    q, k = torch.zeros((2, 3, 4, 64), dtype=BF16, device="cuda"), torch.zeros((2, 3, 2, 64), dtype=BF16, device="cuda")
    freqs, pos = freqs_of(64).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def refused(err=ValueError, q=q, k=k, freqs=freqs, positions=pos, **kw):
        with pytest.raises(err):
            rsv.rotate_tokens(q, k, freqs, positions, **kw)
    refused(q=q.float())
    refused(k=k[:1])
    refused(k=k[..., :32])
    refused(freqs=freqs.double())
    refused(freqs=torch.zeros(33, device="cuda"))
    refused(freqs=freqs[:0])
    refused(positions=None)
    refused(positions=pos.long())
    refused(axes=torch.zeros(32, **i32))                       # no ids
    refused(ids=torch.zeros((1, 2, 2), **i32))
    refused(ids=torch.zeros((2, 2, 3), **i32), axes=torch.zeros(31, **i32))
    refused(parents=torch.zeros((2, 2), **i32))
    refused(query_lens=torch.zeros(3, **i32))
    refused(q_out=torch.zeros((2, 3, 4, 64), device="cuda"))
    refused(rsv.SpecVerifyError, freqs=freqs[:4])              # 8 channels
    refused(rsv.SpecVerifyError, ids=torch.zeros((17, 2, 3), **i32))
    refused(rsv.SpecVerifyError, q_out=q[:, :, :, :], k_out=q[:, :, :2])
    same = torch.zeros((2, 3, 2, 64), dtype=BF16, device="cuda")
    refused(rsv.SpecVerifyError, q=same, k=k, k_out=same)      # another's input
