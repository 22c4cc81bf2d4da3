"""sample_tokens where a draw falls on a border exactly: uniforms of 0 and on a
running sum, beside logits that weigh nothing.

Draws are exact here: the weights are powers of two, zeros, or far enough
apart that no rounding (2^-38 of a row's mass) reaches a border.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import sample_ref as S

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")
AT_ZERO = [0.0, -1.0, NAN, 2.0 ** -149]


def check(x, T, u, **rules):
    """Rows x [B, V] with the uniforms u; tokens and logprobs start as what no draw gives."""
    B, V = x.shape
    T = float(np.float32(T))
    u = torch.tensor(u).expand(B, 1, len(u)).contiguous()
    tokens = torch.full(u.shape, 77_777_777, dtype=torch.int32, device="cuda")
    logprobs = torch.full(u.shape, 55.0, device="cuda")
    dev = {k: v.cuda() for k, v in rules.items()}
    rsv.sample_tokens(x[:, None].cuda(), u.cuda(), torch.full((B,), T, device="cuda"), tokens=tokens, logprobs=logprobs, **dev)
    for b in range(B):
        ids, w = S.kept(x[b].double().numpy(), T, *(rules[k][b].item() if k in rules else None for k in ("top_k", "top_p", "min_p")))
        w = np.where(w < 2.0 ** -1000, 0.0, w)
        for j in range(u.shape[2]):
            token, lp = S.draw(ids, w, float(u[b, 0, j]))
            assert tokens[b, 0, j] == token, (b, j, float(u[b, 0, j]), int(tokens[b, 0, j]), token)
            assert abs(float(logprobs[b, 0, j]) - lp) <= 2.0 ** -24 * abs(lp) + 1e-9, (b, j)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [700, 5000, 40000, 300000])
def test_masked_tokens_before_a_draw_of_nothing(V, dtype):
    """The first tokens masked, up to all but one: parts of a wave's vectors, whole ones, whole chunks."""
    runs = [n for n in (1, 255, 256, 257, 511, 512, 513, 2048, 2049, 4095, 4096, 16383, 16384, 20000, V - 1) if n < V]
    g = torch.Generator().manual_seed(V)
    x = torch.randn((len(runs), V), generator=g).to(DTYPES[dtype])
    for b, n in enumerate(runs):
        x[b, :n] = -INF
    check(x, 0.8, AT_ZERO + [0.3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 40])
def test_draws_on_a_border_between_chunks(rows, dtype):
    """Two or four equal logits far apart, all others masked: a draw of 0.5 is the first after the border."""
    x = torch.full((4, 50000), -INF)
    x[0, [600, 17001]] = 1.0
    x[1, [5, 49999]] = -3.0
    x[2, [300, 9000, 33000, 49000]] = 0.0
    x[3, [2000, 2001]] = 100.0
    check(x.repeat(rows, 1).to(DTYPES[dtype]), 1.0, AT_ZERO[:3] + [0.5, 0.25, 0.75])


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_that_weigh_nothing_are_not_drawn(dtype):
    """Beside +inf, and so far below the largest that float64 knows no weight of it."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 30000), generator=g).clamp(-4, 4)
    x[0, 700] = INF
    x[1, [20000, 20001]] = INF
    x[2, 25000:] = 3000.0
    x[3, 100:29000] = -INF
    x[3, 29500] = 5000.0
    x[4, :20000] = -2000.0
    check(x.to(DTYPES[dtype]), 1.0, AT_ZERO + [0.5, 0.999])
    check(x.to(DTYPES[dtype]), 1e-3, AT_ZERO + [0.999])
