"""adjust_logits against its formulas in float64, on the GPU.

Tolerance.  The kernel computes in float32 at most one product or quotient,
the product frequency * n, two subtractions and one addition, each rounded to
within 2^-24 of its result; every result is at most S = |l1| + |f| n + |p| +
|bias| in magnitude, so the float32 value is within 5 * 2^-24 S of the exact
one.  The output's rounding adds half a step: eps / 2 of the value (and, next
to zero, nothing more: values here are far from the subnormals).  Logits that
nothing applies to must keep their bits, and -inf must be exactly where the
formulas put it.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import workloads as W
import rejection_sampling_verifier_amd as rsv
from tests.parity import check_rows, check_tree_rows, run_gpu
from tests.test_gpu_tree import run_tree_gpu

pytestmark = pytest.mark.gpu

INT_MIN = -2 ** 31


def path_nodes(par, v):
    """Nodes on v's path without the root; a bad parent starts the path."""
    out = []
    while v > 0:
        out.append(v)
        p = int(par[v])
        if not 0 <= p < v:
            break
        v = p
    return out


def reference(logits, x):
    """(values, magnitudes S, changed) in float64; logits [B, P, V] float64."""
    B, P, V = logits.shape
    out, S = logits.copy(), np.abs(logits)
    changed = np.zeros(logits.shape, bool)
    get = lambda k: None if x.get(k) is None else x[k].cpu().numpy()  # noqa: E731
    hist, hl, pl, tok, par = (get(k) for k in ("history", "history_lens", "prompt_lens", "tokens", "parents"))
    r, a, f = get("repetition"), get("presence"), get("frequency")
    ids, vals, nb = get("bias_ids"), get("bias_values"), get("bias_lens")
    mask, rows = get("mask"), get("mask_rows")
    pen = not (r is None and a is None and f is None)
    for b in range(B):
        seen0, n0 = np.zeros(V, bool), np.zeros(V)
        if pen and hist is not None:
            for j in range(min(max(int(hl[b]), 0), hist.shape[1])):
                t = int(hist[b, j])
                if 0 <= t < V:
                    seen0[t] = True
                    if pl is None or j >= max(int(pl[b]), 0):
                        n0[t] += 1
        bias = {}
        if ids is not None:
            for e in range(min(max(int(nb[b]), 0), ids.shape[1]) if nb is not None else ids.shape[1]):
                if 0 <= ids[b, e] < V:
                    bias[int(ids[b, e])] = float(vals[b, e])
        for i in range(P):
            seen, n = seen0.copy(), n0.copy()
            if pen and tok is not None and P > 1:
                for t in (tok[b, :i] if par is None else [tok[b, v] for v in path_nodes(par[b], i)]):
                    if 0 <= t < V:
                        seen[t] = True
                        n[t] += 1
            l = out[b, i]
            if pen:
                rr, aa, ff = (d if y is None else float(y[b]) for y, d in ((r, 1.0), (a, 0.0), (f, 0.0)))
                with np.errstate(invalid="ignore"):
                    l[seen] = np.where(l[seen] > 0, l[seen] / rr, l[seen] * rr)
                    S[b, i] = np.abs(l) + abs(ff) * n + abs(aa) * (n > 0)
                    l[n > 0] = (l - ff * n - aa)[n > 0]
                changed[b, i] |= seen
            for t, v in bias.items():
                l[t] += v
                S[b, i, t] += abs(v)
                changed[b, i, t] = True
            if mask is not None:
                row = b * P + i if rows is None else int(rows[b, i])
                if 0 <= row < mask.shape[0]:
                    bits = np.unpackbits(mask[row].view(np.uint8), bitorder="little")[:V].astype(bool)
                    l[~bits] = -np.inf
                    changed[b, i] |= ~bits
    return out, S, changed


def check(logits, x, got):
    ref, S, changed = reference(logits.double().cpu().numpy(), x)
    out = got.double().cpu().numpy()
    eps = torch.finfo(logits.dtype).eps
    np.testing.assert_array_equal(np.isneginf(out), np.isneginf(ref))
    np.testing.assert_array_equal(np.isposinf(out), np.isposinf(ref))
    np.testing.assert_array_equal(np.isnan(out), np.isnan(ref))
    ok = np.isfinite(ref)
    err, tol = np.abs(out - ref)[ok], (np.abs(ref) * eps / 2 + 5 * 2.0 ** -24 * S)[ok]
    assert (err <= tol * (1 + 2.0 ** -20)).all(), float((err - tol).max())
    view = torch.int16 if logits.dtype == torch.bfloat16 else torch.int32
    same = torch.from_numpy(~changed)
    assert torch.equal(got.contiguous().view(view).cpu()[same], logits.contiguous().view(view).cpu()[same])


def make(seed, B, P, V, dtype, hist=40, bias=0, mask=False, pen=True, tree=False, R=3, ids_below=None):
    """Random inputs with bad tokens, bad ids, repeated ids and odd lengths among them."""
    rng = np.random.default_rng(seed)
    top = ids_below or min(V, 60)   # few ids, so that they repeat
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731

    def ids(shape):
        a = rng.integers(0, top, shape)
        bad = rng.random(shape) < 0.1
        return np.where(bad, rng.choice([-1, V, INT_MIN, 2 ** 31 - 1, V + 5], shape), a)

    x = dict(tokens=t(ids((B, P)), torch.int32))
    if pen:
        x["repetition"] = t(rng.uniform(0.7, 1.5, B), torch.float32)
        x["presence"] = t(rng.uniform(-1, 1, B), torch.float32)
        x["frequency"] = t(rng.uniform(-0.5, 0.5, B), torch.float32)
    if hist:
        x["history"] = t(ids((B, hist)), torch.int32)
        lens = rng.integers(-2, hist + 3, B)
        lens[0] = hist
        x["history_lens"] = t(lens, torch.int32)
        x["prompt_lens"] = t(rng.integers(-1, hist + 2, B), torch.int32)
    if tree:
        par = np.array([[rng.integers(max(0, c - 4), c) if c else 0 for c in range(P)] for _ in range(B)])
        if P > 3:
            par[-1, 2] = 2      # not an earlier node
            par[-1, 3] = -7
        x["parents"] = t(par, torch.int32)
    if bias:
        x["bias_ids"] = t(ids((B, bias)), torch.int32)
        x["bias_values"] = t(rng.normal(0, 4, (B, bias)), torch.float32)
        x["bias_lens"] = t(rng.integers(-1, bias + 2, B), torch.int32)
    if mask:
        words = (V + 31) // 32
        m = rng.integers(-2 ** 31, 2 ** 31, (R, words))
        m[0] = 0                # nothing is allowed
        m[1] = np.where(rng.random(words) < 0.5, -1, m[1])
        x["mask"] = t(m, torch.int32)
        x["mask_rows"] = t(rng.integers(-1, R + 1, (B, P)), torch.int32)
    logits = t(rng.normal(0, 3, (B, P, V)), torch.float32)
    logits[torch.rand(logits.shape, device="cuda") < 0.01] = float("-inf")
    return logits.to(dtype), x


DT = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 64, 4095, 4096, 4097, 4104, 8195, 12288, 20001])
def test_every_control_over_vocabulary_sizes(V, dtype):
    logits, x = make(V, 3, 4, V, dtype, bias=9, mask=True)
    check(logits, x, rsv.adjust_logits(logits, **x))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("pen", [False, True])
@pytest.mark.parametrize("bias", [0, 1, 70])
@pytest.mark.parametrize("mask", [False, True])
def test_each_control_by_itself(dtype, pen, bias, mask):
    logits, x = make(5, 2, 3, 5003, dtype, pen=pen, bias=bias, mask=mask)
    check(logits, x, rsv.adjust_logits(logits, **x))


@pytest.mark.parametrize("leave", ["repetition", "presence", "frequency", "history", "tokens", "prompt_lens", "bias_lens"])
def test_members_left_out(leave):
    P = 1 if leave == "tokens" else 3
    logits, x = make(6, 2, P, 900, torch.float32, bias=5)
    x[leave] = None
    if leave == "history":
        x["history_lens"] = x["prompt_lens"] = None
    check(logits, x, rsv.adjust_logits(logits, **x))


@pytest.mark.parametrize("P", [1, 2, 64, 65])
def test_chains_up_to_the_longest(P):
    logits, x = make(7, 2, P, 300, torch.float32, hist=3)
    check(logits, x, rsv.adjust_logits(logits, **x))
    y = dict(x, tokens=x["tokens"][:, :max(1, P - 1)].contiguous())   # spec_verify's draft_tokens: K of K + 1
    assert torch.equal(rsv.adjust_logits(logits, **y), rsv.adjust_logits(logits, **x))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N", [1, 2, 5, 33, 64])
def test_trees(N, dtype):
    logits, x = make(8 + N, 3, N, 700, dtype, tree=True, bias=3, mask=True, ids_below=20)
    check(logits, x, rsv.adjust_logits(logits, **x))


def test_a_chain_given_as_a_tree_is_the_chain():
    B, P, V = 2, 20, 1000
    logits, x = make(9, B, P, V, torch.float32)
    tree = dict(x, parents=(torch.arange(P, dtype=torch.int32) - 1).expand(B, P).contiguous().cuda(),
                tokens=torch.cat([x["tokens"][:, :1] * 0 + 5, x["tokens"][:, :P - 1]], 1).contiguous())
    assert torch.equal(rsv.adjust_logits(logits, **x), rsv.adjust_logits(logits, **tree))


@pytest.mark.parametrize("dtype", DT)
def test_long_histories_count_exactly(dtype):
    logits, x = make(10, 2, 2, 9000, dtype, hist=70001, ids_below=9000)
    check(logits, x, rsv.adjust_logits(logits, **x))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V, pitch, shift", [(4097, 4100, 0), (1001, 1001, 1), (5000, 5003, 3), (777, 1024, 5)])
def test_strided_views_in_place_and_out_of_place(V, pitch, shift, dtype):
    """Any element alignment; what lies between the rows keeps its bits; in place gives the same bits."""
    B, P = 3, 4
    logits, x = make(11, B, P, V, dtype, bias=6, mask=True)
    flat = torch.full((shift + B * (P + 1) * pitch,), 7.0, dtype=dtype, device="cuda")
    view = flat[shift:].view(B, P + 1, pitch)[:, :P, :V]     # target[:, :K] of a padded vocabulary
    view.copy_(logits)
    want = rsv.adjust_logits(logits, **x)
    check(logits, x, want)
    assert torch.equal(rsv.adjust_logits(view, **x).nan_to_num(), want.nan_to_num())
    assert torch.equal(view, logits)
    assert rsv.adjust_logits(view, out=view, **x) is view
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(view.contiguous().view(bits), want.view(bits))
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep[shift:].view(B, P + 1, pitch)[:, :P, :V] = False
    assert (flat[keep] == 7.0).all()


@pytest.mark.parametrize("dtype", DT)
def test_infinities_and_nan_pass_by_their_own_tokens_only(dtype):
    logits, x = make(12, 2, 2, 600, dtype, bias=4, mask=True)
    logits[:, :, 1] = float("nan")
    logits[:, :, 2] = float("inf")
    logits[:, :, 3] = float("-inf")
    logits[:, :, 4] = torch.finfo(dtype).min
    x["mask_rows"][0, 0] = 0                       # all forbidden, NaN among them
    x["mask_rows"][1] = -1
    out = rsv.adjust_logits(logits, **x)
    assert torch.isneginf(out[0, 0]).all()
    check(logits, x, out)


def test_masks_without_rows_go_by_position():
    logits, x = make(13, 3, 2, 100, torch.float32, mask=True, R=6)
    x["mask_rows"] = None
    check(logits, x, rsv.adjust_logits(logits, **x))


def test_many_rows_and_one_group_of_positions():
    logits, x = make(14, 600, 3, 4500, torch.bfloat16, bias=3, mask=True, hist=6)
    check(logits, x, rsv.adjust_logits(logits, **x))


def test_side_stream_and_graph_replays():
    sets = [make(20 + i, 2, 3, 5000, torch.bfloat16, bias=5, mask=True) for i in range(3)]
    static_l = sets[0][0].clone()
    static = {k: v.clone() for k, v in sets[0][1].items()}
    out = torch.empty_like(static_l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rsv.adjust_logits(static_l, out=out, **static)
        fresh = rsv.adjust_logits(static_l, **static)
    torch.cuda.synchronize()
    assert torch.equal(out, fresh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rsv.adjust_logits(static_l, out=out, **static)
    for i in (1, 2, 0, 1, 1):
        static_l.copy_(sets[i][0])
        for k, v in sets[i][1].items():
            static[k].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rsv.adjust_logits(sets[i][0], **sets[i][1])), i


def _as_numpy(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("topk", [0, 64])
def test_adjusted_logits_verified_as_a_chain(topk):
    """As a program uses it: both logit sets adjusted, then verified; the oracle verifies the adjusted logits."""
    d = W.make(W.Case(B=4, K=5, V=9001, dtype=W.BF16, draft_sigma=0.7, temperature=0.8, greedy_rows=1, topk=topk,
                      seed=77))
    B, K, V = d["draft"].shape
    tgt, dft = (torch.from_numpy(d[k]).view(torch.bfloat16).cuda() for k in ("target", "draft"))
    _, x = make(30, B, K + 1, V, torch.bfloat16, hist=50, bias=8, ids_below=V)
    x["tokens"] = torch.from_numpy(d["tokens"].astype(np.int32)).cuda()
    check(tgt, x, rsv.adjust_logits(tgt, **x))
    check(dft, x, rsv.adjust_logits(dft, **x))
    e = dict(d, target=_as_numpy(rsv.adjust_logits(tgt, **x)), draft=_as_numpy(rsv.adjust_logits(dft, **x)))
    check_rows(e, run_gpu(e))


def test_adjusted_logits_verified_as_a_tree():
    d = W.make_tree(W.TreeCase(B=3, V=7000, dtype=W.BF16, draft_sigma=1.0, temperature=1.0,
                               parents=W.level_tree((3, 4, 3)), topk=0, seed=78))
    B, N, V = d["target"].shape
    tgt, dft = (torch.from_numpy(d[k]).view(torch.bfloat16).cuda() for k in ("target", "draft"))
    _, x = make(31, B, N, V, torch.bfloat16, hist=50, bias=8, ids_below=V)
    x["tokens"] = torch.from_numpy(d["tokens"].astype(np.int32)).cuda()
    x["parents"] = torch.from_numpy(np.broadcast_to(d["parents"], (B, N)).astype(np.int32).copy()).cuda()
    e = dict(d, target=_as_numpy(rsv.adjust_logits(tgt, **x)), draft=_as_numpy(rsv.adjust_logits(dft, **x)))
    check_tree_rows(e, run_tree_gpu(e))


def test_refusals_on_device_tensors():
    logits, x = make(15, 2, 3, 100, torch.float32, bias=4, mask=True)
    def refused(err=ValueError, logits=logits, **kw):  # noqa: E306
        with pytest.raises(err):
            rsv.adjust_logits(logits, **dict(x, **kw))
    refused(tokens=x["tokens"][:, :1])
    refused(tokens=x["tokens"].long())
    refused(tokens=None)
    refused(history_lens=None)
    refused(parents=x["tokens"][:, :2])
    refused(repetition=x["repetition"].double())
    refused(repetition=x["repetition"].cpu())
    refused(bias_values=x["bias_values"][:, :2].contiguous())
    refused(mask=x["mask"][:, :2].contiguous())
    refused(mask_rows=None)
    refused(out=logits[:, :2])
    refused(out=logits.bfloat16())
    refused(logits=logits.transpose(1, 2))
    refused(logits=logits[:, :1].expand(2, 3, 100))
    refused(logits=logits[0])
    refused(TypeError, logits=logits.half())
    refused(logits=torch.empty((2, 3, 0), device="cuda"))
    big = torch.zeros((2, 3, 200), device="cuda")
    with pytest.raises(rsv.SpecVerifyError):     # overlaps its input, shifted
        rsv.adjust_logits(big[:, :, :100], **dict(x, out=big[:, :, 50:150]))
    with pytest.raises(rsv.SpecVerifyError):
        rsv.adjust_logits(torch.zeros((2, 66, 100), device="cuda"), torch.zeros((2, 66), dtype=torch.int32, device="cuda"),
                          repetition=x["repetition"])
