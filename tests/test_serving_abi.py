"""Argument checks of the operators around a verification step, on the host:
every call here returns before it launches anything."""

from __future__ import annotations

import ctypes

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding as B

A = 0x10000000                 # made-up device addresses, far apart
P = [A + (i << 32) for i in range(64)]


def adjust(**kw):
    a = dict(logits=P[0], row=3000, stride=1000, tokens=P[1], tok_stride=2, parents=None, c=B.SvControls(), B=2, P=3,
             V=1000, dtype=B.SV_BF16, out=P[2], out_row=3000, out_stride=1000)
    c = {k[2:]: kw.pop(k) for k in list(kw) if k.startswith("c_")}
    a.update(kw)
    for k, v in c.items():
        setattr(a["c"], k, v)
    return B.load_library().spec_verify_adjust_logits(
        a["logits"], a["row"], a["stride"], a["tokens"], a["tok_stride"], a["parents"],
        ctypes.byref(a["c"]) if a["c"] is not None else None, a["B"], a["P"], a["V"], a["dtype"], a["out"],
        a["out_row"], a["out_stride"], None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(out=None), dict(c=None), dict(B=0), dict(P=0), dict(V=0), dict(dtype=2), dict(dtype=-1),
    dict(stride=999), dict(out_stride=999), dict(row=2999), dict(out_row=2999), dict(stride=2 ** 60),
    dict(row=2 ** 60), dict(logits=P[0] + 1), dict(out=P[2] + 1),
    dict(out=P[0] + 2), dict(out=P[0], out_row=3001), dict(out=P[0] + 2 * 5998),            # overlaps
    dict(c_repetition=P[3], tokens=None), dict(c_presence=P[3], tok_stride=1),
    dict(c_frequency=P[3], parents=P[4], tok_stride=2),
    dict(c_repetition=P[3], c_history=P[5], c_history_stride=4),                             # no lengths
    dict(c_repetition=P[3], c_history=P[5], c_history_lens=P[6], c_history_stride=-1),
    dict(c_bias_ids=P[7]), dict(c_bias_ids=P[7], c_bias_values=P[8], c_bias_stride=-1),
    dict(c_mask=P[9], c_num_masks=-1), dict(c_mask=P[9], c_num_masks=5),                     # fewer than B P, no rows
])
def test_adjust_logits_refuses(bad):
    assert adjust(**bad) == B.SV_ERR_ARG


def test_adjust_logits_limits():
    assert adjust(P=B.SV_MAX_K + 2, row=1 << 20, out_row=1 << 20) == B.SV_ERR_UNSUPPORTED
    assert adjust(P=B.SV_MAX_NODES + 1, parents=P[4], row=1 << 20, out_row=1 << 20) == B.SV_ERR_UNSUPPORTED
    assert adjust(B=2 ** 31 - 1, P=1, V=5000, row=5000, stride=5000, out_row=5000, out_stride=5000,
                  out=P[0] + (1 << 50)) == B.SV_ERR_UNSUPPORTED


def test_adjust_logits_takes_gpu_tensors_only():
    with pytest.raises(ValueError):
        rsv.adjust_logits(torch.zeros(1, 1, 8))
    with pytest.raises(ValueError):
        rsv.adjust_logits(None)


def cache(**kw):
    c = B.SvCache(P[0], P[1], P[2], P[3], P[4], P[5], P[6], 2, 100, 2, 64, 16, 10, 32, B.SV_E4M3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attention(ws=P[20], ws_n=None, **kw):
    a = dict(q=P[10], q_row=3 * 512, q_tok=512, kn=P[11], vn=P[12], kv_row=3 * 512, kv_tok=512, c=cache(),
             positions=P[13], blocks=P[14], parents=None, lens=None, T=3, H=4, scale=0.125, out=P[15], weights=None)
    a.update(kw)
    n = ctypes.c_size_t(1 << 40 if ws_n is None else ws_n)
    rc = B.load_library().spec_verify_attention(
        a["q"], a["q_row"], a["q_tok"], a["kn"], a["vn"], a["kv_row"], a["kv_tok"],
        None if a["c"] is None else ctypes.byref(a["c"]), a["positions"], a["blocks"], a["parents"], a["lens"], a["T"],
        a["H"], a["scale"], a["out"], a["weights"], ws, ctypes.byref(n), None)
    return rc if ws is not None else (rc, n.value)


BAD_CACHES = [dict(k_pages=None), dict(v_pages=None), dict(k_scale=None), dict(v_scale=None), dict(k_tail=None),
              dict(v_tail=None), dict(block_table=None), dict(B=0), dict(num_pages=0), dict(Hkv=0), dict(max_blocks=0),
              dict(page=0), dict(tail=0), dict(kind=2), dict(tail=24), dict(k_pages=P[0] + 8), dict(v_tail=P[5] + 2),
              dict(k_scale=P[2] + 2), dict(block_table=P[6] + 1)]
UNSUPPORTED_CACHES = [dict(D=32), dict(D=96), dict(D=256), dict(page=8, tail=32), dict(page=48, tail=48),
                      dict(page=512, tail=512), dict(Hkv=5000), dict(max_blocks=B.SV_MAX_BLOCKS + 1),
                      dict(B=70000)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_attention_refuses_bad_caches(bad):
    assert attention(c=cache(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", UNSUPPORTED_CACHES)
def test_attention_refuses_unsupported_caches(bad):
    assert attention(c=cache(**bad)) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(c=None), dict(q=None), dict(kn=None), dict(vn=None), dict(positions=None), dict(blocks=None), dict(out=None),
    dict(T=0), dict(H=0), dict(H=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(q=P[10] + 8), dict(kn=P[11] + 2), dict(out=P[15] + 8), dict(q_tok=516),
    dict(kv_row=-8), dict(q_row=1 << 50), dict(weights=P[16] + 2), dict(ws=P[20] + 16)])
def test_attention_refuses(bad):
    assert attention(**bad) == B.SV_ERR_ARG


ROW = 2 * 3 * 512               # bytes from one row of q, k_new and v_new to the next;
QB, KB = 2048 + 512, 2048 + 256  # of a row that are read; of the outputs:
OUT, WEIGHTS = 2 * 2 * 3 * 4 * 64, 2 * 3 * 10 * 4


@pytest.mark.parametrize("bad", [
    dict(out=P[10]), dict(out=P[10] + QB - 16), dict(out=P[10] + ROW + QB - 16), dict(out=P[10] + 16 - OUT),
    dict(out=P[11]), dict(out=P[11] + KB - 16), dict(out=P[12] + ROW + KB - 16), dict(out=P[12] + 16 - OUT),
    dict(q_row=0, out=P[10] + QB - 16), dict(weights=P[10]), dict(weights=P[12] + KB - 4),
    dict(weights=P[11] + 4 - WEIGHTS), dict(weights=P[15]), dict(weights=P[15] + OUT - 4),
    dict(weights=P[15] + 4 - WEIGHTS)])
def test_attention_refuses_outputs_over_what_it_reads(bad):
    assert attention(**bad) == B.SV_ERR_ARG


def test_attention_limits_and_workspace():
    assert attention(T=B.SV_MAX_K + 2) == B.SV_ERR_UNSUPPORTED
    assert attention(T=B.SV_MAX_NODES + 1, parents=P[16]) == B.SV_ERR_UNSUPPORTED
    assert attention(H=2 * 257) == B.SV_ERR_UNSUPPORTED
    rc, n = attention(ws=None)
    assert rc == B.SV_OK and n > 0 and n % 256 == 0
    rc, more = attention(ws=None, weights=P[16])
    assert rc == B.SV_OK and more > n
    assert attention(ws_n=n - 1) == B.SV_ERR_WORKSPACE
    assert attention(weights=P[16], ws_n=n) == B.SV_ERR_WORKSPACE


def test_cache_attention_takes_gpu_tensors_only():
    with pytest.raises(ValueError):
        rsv.KVCache(*(torch.zeros(1, 1, 16, 64, dtype=torch.uint8),) * 7)
    with pytest.raises(ValueError):
        rsv.new_cache(1, 1, 1, 64, device="cpu")


def commit(**kw):
    a = dict(kn=P[10], vn=P[11], kv_row=3 * 512, kv_tok=512, T=3, num=P[12], nodes=None, stride=0, c=cache(),
             positions=P[13], blocks=P[14], positions_out=P[15], blocks_out=P[16], weights=None, totals=None,
             totals_out=None)
    a.update(kw)
    if a["c"] is not None:
        a["c"] = ctypes.byref(a["c"])
    return B.load_library().spec_verify_commit(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_CACHES + [dict(tail=16)])   # 16 slots, and 15 + 3 tokens
def test_commit_refuses_bad_caches(bad):
    assert commit(c=cache(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", UNSUPPORTED_CACHES)
def test_commit_refuses_unsupported_caches(bad):
    assert commit(c=cache(**bad)) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(c=None), dict(kn=None), dict(vn=None), dict(num=None), dict(positions=None), dict(blocks=None),
    dict(positions_out=None), dict(blocks_out=None), dict(T=0), dict(kn=P[10] + 8), dict(kv_tok=4), dict(kv_row=-8),
    dict(positions_out=P[13]), dict(blocks_out=P[14]), dict(positions_out=P[16]), dict(positions_out=P[14]),
    dict(positions_out=P[13] + 4), dict(blocks_out=P[14] + 4), dict(nodes=P[17], stride=1),
    dict(positions_out=P[12]), dict(blocks_out=P[12] - 4),
    dict(weights=P[18]), dict(totals=P[18]), dict(totals_out=P[18]), dict(totals=P[18], totals_out=P[18] + 40)])
def test_commit_refuses(bad):
    assert commit(**bad) == B.SV_ERR_ARG


def test_commit_limits():
    assert commit(T=B.SV_MAX_K + 2, c=cache(tail=128)) == B.SV_ERR_UNSUPPORTED


def evict(**kw):
    a = dict(totals=P[0], table=P[1], blocks=P[2], B=4, most=100, budget=10, first=1, last=1, totals_out=P[3],
             table_out=P[4], blocks_out=P[5], evicted=P[6])
    a.update(kw)
    return B.load_library().spec_verify_evict(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(totals=None), dict(table=None), dict(blocks=None), dict(totals_out=None), dict(table_out=None),
    dict(blocks_out=None), dict(evicted=None), dict(B=0), dict(most=0), dict(budget=-1), dict(first=-1), dict(last=-1),
    dict(totals_out=P[0] + 4), dict(table_out=P[1] + 400), dict(totals_out=P[1]), dict(table_out=P[0]),
    dict(table_out=P[3] + 8), dict(blocks_out=P[2] + 4), dict(evicted=P[2]), dict(evicted=P[5] + 12)])
def test_evict_refuses(bad):
    assert evict(**bad) == B.SV_ERR_ARG


def test_evict_limits():
    assert evict(most=B.SV_MAX_BLOCKS + 1) == B.SV_ERR_UNSUPPORTED
    assert evict(most=16385, table_out=P[1]) == B.SV_ERR_UNSUPPORTED   # in place, beyond what LDS can hold
