"""sample_tokens and truncate_logits against their definitions in 64 bits, on
the GPU.

Tokens and kept sets are compared exactly.  The masses that decide are off by at
most 2^-44 of the largest weight for each kept token (their rounding to 2^-43)
plus a few 2^-50 of each weight: a draw's token can differ only where u times
the mass lies that near a border, for which the cases' seeds leave a chance
below 10^-6.  A logprob is rounded to float32 (2^-24 of it) from an error below
10^-9.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import sample_ref as S

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def logits_of(seed, B, P, V, dtype, sigma=3.0, peaks=20, grid=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, P, V), generator=g) * sigma
    if peaks:
        x.scatter_add_(2, torch.randint(0, V, (B, P, peaks), generator=g), torch.full((B, P, peaks), 8.0))
    if grid:
        x = (x / grid).round() * grid
    return x.to(DTYPES[dtype])


def rules(B, **kw):
    out = {}
    for name, dt in (("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32)):
        v = kw.get(name)
        if v is not None:
            out[name] = torch.tensor([v[b % len(v)] for b in range(B)] if isinstance(v, list) else [v] * B, dtype=dt)
    return out


def check(x, T, u, **kw):
    """x [B, P, V] on the CPU (any strides that the call takes)."""
    B, P, V = x.shape
    n = u.shape[2]
    T = torch.tensor([T[b % len(T)] for b in range(B)] if isinstance(T, list) else [T] * B, dtype=torch.float32)
    r = rules(B, **kw)
    base = x._base if x._base is not None else x
    gpu = torch.as_strided(base.cuda(), x.size(), x.stride(), x.storage_offset())
    dev = {k: v.cuda() for k, v in r.items()}
    tokens, logprobs = rsv.sample_tokens(gpu, u.cuda(), T.cuda(), logprobs=True, **dev)
    cut = rsv.truncate_logits(gpu, T.cuda(), **dev)
    tokens, logprobs, cut = tokens.cpu().numpy(), logprobs.cpu().numpy(), cut.cpu()
    for b in range(B):
        args = [None if k not in r else r[k][b].item() for k in ("top_k", "top_p", "min_p")]
        for i in range(P):
            row = x[b, i].double().numpy()
            bits = x[b, i].contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)
            got = cut[b, i].view(bits.dtype)
            if not float(T[b]) > 0:
                want = [S.greedy(row)] * n
                assert torch.equal(got, bits)
            else:
                ids, w = S.kept(row, float(T[b]), *args)
                want = [S.draw(ids, w, float(u[b, i, j])) for j in range(n)]
                finite = int(np.sum(row > -np.inf))
                if len(ids) == finite:
                    same = torch.from_numpy(~np.isnan(row))
                    assert torch.equal(got[same], bits[same]), (b, i)
                else:
                    left = torch.zeros(V, dtype=torch.bool)
                    left[torch.from_numpy(ids)] = True
                    assert torch.equal(got[left], bits[left]), (b, i)
                    wrong = (cut[b, i][~left] != -np.inf).nonzero().flatten().tolist()
                    assert not wrong, (b, i, args, wrong[:5], len(ids))
            for j in range(n):
                assert tokens[b, i, j] == want[j][0], (b, i, j, args, float(u[b, i, j]))
                assert (logprobs[b, i, j] == want[j][1]
                        or abs(logprobs[b, i, j] - want[j][1]) <= 2.0 ** -24 * abs(want[j][1]) + 1e-9)
    # in place: the same
    rsv.truncate_logits(gpu, T.cuda(), out=gpu, **dev)
    torch.testing.assert_close(gpu.cpu(), cut, rtol=0, atol=0, equal_nan=True)
    if base.numel() > x.numel():
        after = torch.as_strided(gpu, base.size(), base.stride(), 0).cpu()
        torch.as_strided(after, x.size(), x.stride(), x.storage_offset()).copy_(x)
        assert torch.equal(after.view(torch.uint8), base.view(torch.uint8))


def uniforms(seed, B, P, n):
    return torch.rand((B, P, n), generator=torch.Generator().manual_seed(seed))


MIX = dict(top_k=[0, 5, 50, 1, 40], top_p=[0.9, 1.0, 0.5], min_p=[0.0, 0.05])
KINDS = {"none": {}, "k": dict(top_k=[50, 1, 0, 130]), "p": dict(top_p=[0.9, 0.3, 1.0]), "m": dict(min_p=[0.1, 0.0, 0.9]),
         "all": MIX}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 512, 1000, 4096, 4097, 32003])
def test_vocabularies(V, dtype, kind):
    check(logits_of(V, 3, 2, V, dtype), [0.8, 1.0, 0.0], uniforms(V + 1, 3, 2, 3), **KINDS[kind])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_full_vocabulary(dtype, kind):
    check(logits_of(1, 4, 1, 151936, dtype), [0.7, 1.0, 0.9, 0.0], uniforms(2, 4, 1, 2), **KINDS[kind])


@pytest.mark.parametrize("kind", ["none", "k", "p", "all"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_enough_rows_for_large_chunks(dtype, kind):
    """Batches that take chunks of eight vectors a thread."""
    check(logits_of(3, 300, 2, 32003 if dtype == "bf16" else 20001, dtype), [0.8, 1.0, 0.6], uniforms(4, 300, 2, 1), **KINDS[kind])


@pytest.mark.parametrize("kind", ["none", "k", "p"])
def test_the_largest_vocabulary(kind):
    check(logits_of(5, 1, 1, 1 << 20, "f32"), 0.9, uniforms(6, 1, 1, 2), **KINDS[kind])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lead", [1, 3, 4])
def test_odd_strides_and_alignments(lead, dtype, kind):
    store = logits_of(7, 3, 2, 5003, dtype)
    check(store[:, :, lead:lead + 4990], 0.8, uniforms(8, 3, 2, 2), **KINDS[kind])


@pytest.mark.parametrize("sigma", [0.0, 0.3])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rule", [dict(top_p=[0.9, 0.999, 0.0]), dict(top_k=[7000, 20000, 999]), dict(min_p=[0.2, 1.0, 1e-6]),
                                  dict(top_k=[30000, 6000], top_p=[0.7, 0.99])])
def test_flat_logits(rule, dtype, sigma):
    """More candidates than lists and LDS hold; with sigma 0 all logits are equal and ids alone decide."""
    check(logits_of(9, 3, 1, 60001, dtype, sigma=sigma, peaks=0), 1.0, uniforms(10, 3, 1, 3), **rule)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("grid", [0.5, 4.0])
def test_cuts_between_equal_logits(grid, dtype):
    x = logits_of(11, 6, 2, 9000, dtype, grid=grid)
    for rule in (dict(top_k=[1, 2, 30, 500, 3000, 8999]), dict(top_p=[0.01, 0.2, 0.5, 0.77, 0.95, 0.99]),
                 dict(top_k=[1, 2, 30, 500, 3000, 8999], top_p=[0.5, 0.9], min_p=[0.0, 0.01, 0.5])):
        check(x, [1.0, 2.0, 0.5], uniforms(12, 6, 2, 4), **rule)


def test_rules_at_their_ends():
    x = logits_of(13, 12, 1, 3000, "f32")
    u = uniforms(14, 12, 1, 2)
    inf, nan = float("inf"), float("nan")
    check(x, 0.8, u, top_k=[-1, 0, 1, 2999, 3000, 3001, 2 ** 31 - 1, -2 ** 31])
    check(x, 0.8, u, top_p=[0.0, -1.0, -inf, 1.0, 1.5, inf, nan, 1e-30, 0.99999994])
    check(x, 0.8, u, min_p=[0.0, -1.0, 1.0, 1.5, inf, nan, 1e-30, 1e-45, 0.99999994])
    check(x, [1e-30, 1e-45, 1e30, inf, 0.0, -1.0, nan, -inf, 1e-3, 50.0], u, top_k=[5, 0], top_p=[0.9, 1.0, 0.5])
    check(x, [1e-30, 1e-45, 1e30, inf, 0.0, -1.0, nan, -inf, 1e-3, 50.0], u)


def test_uniforms_at_their_ends():
    x = logits_of(15, 3, 1, 2000, "bf16")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan"), 2.0 ** -149, 0.5]).expand(3, 1, 8).contiguous()
    for kind in KINDS.values():
        check(x, 0.8, u, **kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan(dtype, kind):
    inf, nan = float("inf"), float("nan")
    x = logits_of(17, 8, 1, 5000, dtype)
    x[0, 0, ::2] = -inf
    x[1, 0, 5:4990] = -inf
    x[2, 0, :] = -inf                    # nothing is left
    x[3, 0, 100] = inf
    x[4, 0, [7, 3000]] = inf
    x[5, 0, ::3] = nan
    x[6, 0, :] = nan
    x[7, 0, :] = -inf
    x[7, 0, 4999] = -3e38
    check(x, 0.8, uniforms(18, 8, 1, 2), **KINDS[kind])
    check(x, 0.0, uniforms(18, 8, 1, 2), **KINDS[kind])


def test_zeros_of_both_signs_are_equal():
    x = torch.zeros((2, 1, 600))
    x[0, 0, ::2] = -0.0
    check(x, 1.0, uniforms(19, 2, 1, 5), top_k=[300, 7])
    check(x.bfloat16(), 1.0, uniforms(19, 2, 1, 5), top_p=[0.4, 0.01])


@pytest.mark.parametrize("kind", ["none", "all"])
def test_up_to_64_draws(kind):
    check(logits_of(21, 2, 2, 30000, "bf16"), 1.0, uniforms(22, 2, 2, 64), **KINDS[kind])


def test_workspaces_need_no_clearing():
    x, u = logits_of(23, 4, 3, 20000, "bf16").cuda(), uniforms(24, 4, 3, 2).cuda()
    T = torch.full((4,), 0.8, device="cuda")
    r = {k: v.cuda() for k, v in rules(4, **MIX).items()}
    want = rsv.sample_tokens(x, u, T, logprobs=True, **r)
    ws = torch.full((rsv.sample_workspace_bytes(4, 3, 20000),), 0xFF, dtype=torch.uint8, device="cuda")
    got = rsv.sample_tokens(x, u, T, logprobs=True, workspace=ws, **r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    cut = rsv.truncate_logits(x, T, **r)
    ws = torch.full((rsv.truncate_workspace_bytes(4, 3, 20000),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(rsv.truncate_logits(x, T, workspace=ws, **r), cut)


def test_graphs_and_streams():
    """Replays over inputs changed in place; two streams at once."""
    B, P, V, n = 5, 3, 40000, 2
    x, u = logits_of(25, B, P, V, "bf16").cuda(), uniforms(26, B, P, n).cuda()
    T = torch.full((B,), 0.8, device="cuda")
    r = {k: v.cuda() for k, v in rules(B, **MIX).items()}
    tokens, lp = torch.zeros((B, P, n), dtype=torch.int32, device="cuda"), torch.zeros((B, P, n), device="cuda")
    out = torch.empty_like(x)

    def step():
        rsv.sample_tokens(x, u, T, tokens=tokens, logprobs=lp, **r)
        rsv.truncate_logits(x, T, out=out, **r)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(logits_of(30 + i, B, P, V, "bf16"))
        u.copy_(uniforms(40 + i, B, P, n))
        T.fill_(0.5 + 0.2 * i)
        want, wlp = rsv.sample_tokens(x, u, T, logprobs=True, **r)
        wout = rsv.truncate_logits(x, T, **r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, want) and torch.equal(lp, wlp) and torch.equal(out, wout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rsv.sample_tokens(x, u, T, stream=side.cuda_stream, **r)
    here = rsv.sample_tokens(x, u, T, **r)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(here, want)


def test_drafts_drawn_so_are_all_accepted_by_the_same_model():
    """Where target and draft are one distribution every draft is accepted, with top-k drafts of a truncated target too."""
    B, K, V = 6, 4, 20000
    x = logits_of(27, B, K + 1, V, "bf16").cuda()
    T, k = torch.full((B,), 0.9, device="cuda"), torch.full((B,), 40, dtype=torch.int32, device="cuda")
    cut = rsv.truncate_logits(x, T, top_k=k)
    drafts = rsv.sample_tokens(x[:, :K], uniforms(28, B, K, 1).cuda(), T, top_k=k)[:, :, 0].contiguous()
    u = torch.rand((B, K + 1), device="cuda")
    tokens, accepted = rsv.verify(cut, x[:, :K].contiguous(), drafts, u, T, topk_draft=40)
    assert accepted.tolist() == [K] * B and torch.equal(tokens[:, :K], drafts)
    # and a draft that the cut leaves out is rejected
    worst = x[:, :K].float().argmin(2).int()
    _, accepted = rsv.verify(cut, x[:, :K].contiguous(), worst, u, T)
    assert accepted.tolist() == [0] * B


def test_refusals_on_device_tensors():
    x, u = torch.zeros((2, 3, 100), device="cuda"), torch.zeros((2, 3, 1), device="cuda")
    T, k = torch.ones(2, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")

    def refused(err=ValueError, x=x, u=u, T=T, **kw):
        with pytest.raises(err):
            rsv.sample_tokens(x, u, T, **kw)
        kw.pop("tokens", None)
        kw.pop("logprobs", None)
    refused(x=x[0])
    refused(TypeError, x=x.half())
    refused(x=x.transpose(1, 2))
    refused(u=u[:1])
    refused(u=u.double())
    refused(rsv.SpecVerifyError, u=u[:, :, :0])
    refused(rsv.SpecVerifyError, u=torch.zeros((2, 3, 65), device="cuda"))
    refused(T=T[:1])
    refused(top_k=k.long())
    refused(top_p=k)
    refused(min_p=T[:1])
    refused(tokens=torch.zeros((2, 3, 2), dtype=torch.int32, device="cuda"))
    refused(logprobs=u.double())
    refused(rsv.SpecVerifyError, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    refused(rsv.SpecVerifyError, tokens=u.view(torch.int32))
    big = torch.zeros((1, 1, (1 << 20) + 1), device="cuda")
    refused(rsv.SpecVerifyError, x=big, u=u[:1, :1].contiguous(), T=T[:1])
    with pytest.raises(ValueError):
        rsv.truncate_logits(x, T, out=x.double())
    with pytest.raises(rsv.SpecVerifyError):
        rsv.truncate_logits(x[:, :2], T, out=x[:, 1:])
    with pytest.raises(rsv.SpecVerifyError):
        rsv.truncate_logits(x, T, top_p=x.view(-1)[:2], out=x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_nothing_cuts_keep_their_bits(dtype):
    """NaN and zeros of both signs among them, in batches of every size, beside rows that are cut."""
    for B, V in ((3, 3001), (600, 8200)):
        x = logits_of(29, B, 2, V, dtype)
        x[:, :, 5] = float("nan")
        x[:, :, 6] = -float("nan")
        x[:, :, 7:9] = torch.tensor([-0.0, 0.0]).to(x.dtype)
        T = torch.tensor([0.0, 0.9, 0.9] * (B // 3))
        k = torch.tensor([3, 0, 3] * (B // 3), dtype=torch.int32)
        got = rsv.truncate_logits(x.cuda(), T.cuda(), top_k=k.cuda()).cpu()
        bits = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(got[0::3].view(bits), x[0::3].view(bits)) and torch.equal(got[1::3].view(bits), x[1::3].view(bits))
        assert ((got[2::3] > -float("inf")).sum(2) == 3).all()
