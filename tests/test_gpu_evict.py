"""cache_evict against a sort in Python, on the GPU: everything is compared exactly."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R

pytestmark = pytest.mark.gpu


def make(seed, B, most, blocks, ties=0.2):
    g = torch.Generator().manual_seed(seed)
    totals = torch.rand((B, most), generator=g) ** 3 * 50
    totals[torch.rand((B, most), generator=g) < ties] = 0.0
    table = torch.randperm(B * most, generator=g).to(torch.int32).view(B, most)
    return table, totals, torch.tensor(blocks, dtype=torch.int32)


def check(table, totals, blocks, budget, first=0, last=0):
    want = R.evict(table, totals, blocks, budget, first, last)
    got = rsv.cache_evict(table.cuda(), totals.cuda(), blocks.cuda(), budget, keep_first=first, keep_last=last)
    for x, y in zip(got, want):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    if table.shape[1] <= 16384:
        t, s, b = table.cuda(), totals.cuda(), blocks.cuda()
        same = rsv.cache_evict(t, s, b, budget, keep_first=first, keep_last=last, table_out=t, totals_out=s,
                               blocks_out=b)
        assert same[0] is t and same[1] is s and same[2] is b
        for x, y in zip(same, want):
            np.testing.assert_array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("budget", [0, 1, 7, 63, 64, 100, 1000])
@pytest.mark.parametrize("first, last", [(0, 0), (1, 4), (10, 0), (0, 50), (40, 40), (2000, 0), (0, 2 ** 31 - 1)])
def test_budgets_and_kept_ends(budget, first, last):
    check(*make(1, 7, 110, [0, 1, 5, 63, 64, 65, 110]), budget, first, last)


@pytest.mark.parametrize("most", [1, 2, 255, 256, 1023, 1024, 1025, 2049, 8448, 16384, 16385, 40000])
def test_table_sizes(most):
    check(*make(2, 3, most, [most, most // 2, max(1, most - 3)]), most // 3, 1, 2)


@pytest.mark.parametrize("value", [0.0, 1.5, float("inf"), float("nan")])
def test_equal_totals_leave_from_the_front(value):
    table, totals, blocks = make(3, 2, 3000, [3000, 1500])
    totals[:] = value
    check(table, totals, blocks, 700, 3, 5)


def test_odd_totals():
    """Infinities, NaN of either sign, both zeros, negatives and subnormals in order."""
    table, totals, blocks = make(4, 4, 500, [500, 400, 300, 200])
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), -float("nan"), 0.0, -0.0, -3.0, 1e-40, -1e-40, 3e38])
    totals[:, ::3] = odd[torch.arange(167) % 10]
    for budget in (0, 17, 150, 199):
        check(table, totals, blocks, budget)


def test_counts_out_of_range_are_taken_into_it():
    table, totals, blocks = make(5, 3, 64, [-4, 100, 2 ** 31 - 1])
    check(table, totals, blocks, 20, 2, 2)


def test_many_rows():
    check(*make(6, 700, 40, [(7 * b) % 41 for b in range(700)]), 16, 1, 2)


def test_stream_and_graph_replays():
    sets = [make(7 + i, 5, 300, [300, 10, 200, 150, 299]) for i in range(3)]
    static = [x.cuda() for x in sets[0]]
    outs = [torch.empty_like(static[0]), torch.empty_like(static[1]), torch.empty_like(static[2]),
            torch.empty_like(static[2])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(keep_first=1, keep_last=3, table_out=outs[0], totals_out=outs[1], blocks_out=outs[2], evicted=outs[3])
    rsv.cache_evict(*static, 100, stream=side.cuda_stream, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rsv.cache_evict(*static, 100, **kw)
    for i in (1, 2, 0, 1, 1):
        for x, y in zip(static, sets[i]):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, R.evict(*sets[i], 100, 1, 3)):
            np.testing.assert_array_equal(x.cpu().numpy(), y)


def test_refusals_on_device_tensors():
    table, totals, blocks = (x.cuda() for x in make(9, 2, 50, [50, 20]))
    def refused(err=ValueError, table=table, totals=totals, blocks=blocks, budget=10, **kw):  # noqa: E306
        with pytest.raises(err):
            rsv.cache_evict(table, totals, blocks, budget, **kw)
    refused(table=table.long())
    refused(table=table.cpu())
    refused(table=table[:, :0])
    refused(totals=totals[:, :20])
    refused(totals=totals.double())
    refused(blocks=blocks[:1])
    refused(table_out=table.float())
    refused(rsv.SpecVerifyError, budget=-1)
    refused(rsv.SpecVerifyError, keep_first=-1)
    refused(rsv.SpecVerifyError, keep_last=-1)
    refused(rsv.SpecVerifyError, evicted=blocks)
    big = torch.zeros((3, 50), dtype=torch.int32, device="cuda")
    with pytest.raises(rsv.SpecVerifyError):
        rsv.cache_evict(big[:2], totals, blocks, 10, table_out=big[1:])
    wide = torch.zeros((1, 16385), dtype=torch.int32, device="cuda")
    with pytest.raises(rsv.SpecVerifyError):
        rsv.cache_evict(wide, torch.zeros((1, 16385), device="cuda"), blocks[:1].clone(), 10, table_out=wide)
