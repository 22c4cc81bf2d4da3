"""truncate_logits beside NaN: in a row that has a rule NaN becomes -inf, in
every other row it keeps its bits, whatever the batch, in place or not."""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")
# temperature, top_k, top_p, min_p, whether the row has a rule; each leaves every finite logit
ROWS = [(0.9, 50, 1.0, 0.0, True), (0.9, 0, 0.99999994, 0.0, True), (0.9, 0, 1.0, 1e-30, True), (0.9, 50, 0.99999994, 1e-30, True),
        (0.9, 0, 1.0, 0.0, False), (0.9, -3, NAN, NAN, False), (0.0, 50, 0.5, 0.5, False), (0.9, 8200, 2.0, -1.0, False)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [len(ROWS), 600])
def test_nan_beside_rules_that_leave_everything(B, dtype):
    V = 8200
    x = torch.full((B, 2, V), -INF)
    x[:, 0, 100:110] = torch.tensor([1.0, 1.5, 2.0, 1.25, 1.75] * 2)  # near each other: no rule leaves one out
    x[:, 0, ::7] = NAN
    x[:, 0, 5:4000:11] = -NAN
    x[:, 0, 100:110] = torch.tensor([1.0, 1.5, 2.0, 1.25, 1.75] * 2)
    x[:, 1, ::3] = NAN                                               # nothing but NaN and -inf
    x = x.to(DTYPES[dtype])
    x[:, :, 8190] = NAN
    col = lambda i, dt: torch.tensor([ROWS[b % len(ROWS)][i] for b in range(B)], dtype=dt).cuda()  # noqa: E731
    kw = dict(top_k=col(1, torch.int32), top_p=col(2, torch.float32), min_p=col(3, torch.float32))
    T = col(0, torch.float32)
    want = x.clone()
    ruled = torch.tensor([ROWS[b % len(ROWS)][4] for b in range(B)])
    want[ruled] = torch.where(torch.isnan(want[ruled]), torch.full((), -INF, dtype=x.dtype), want[ruled])
    bits = torch.int16 if dtype == "bf16" else torch.int32

    def same(got):
        assert torch.equal(got.cpu().view(bits), want.view(bits))
    g = x.cuda()
    same(rsv.truncate_logits(g, T, **kw))
    odd = torch.zeros((B, 2, V + 9), dtype=x.dtype, device="cuda")[:, :, 3:V + 3]   # other vectors than the logits'
    same(rsv.truncate_logits(g, T, out=odd, **kw).contiguous())
    same(rsv.truncate_logits(g, T, out=g, **kw))
