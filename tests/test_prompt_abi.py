"""Argument checks of the calls that rotate tokens and append prompts, on the
host: every call here returns before it launches anything."""

from __future__ import annotations

import ctypes

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_abi import BAD_CACHES, P, UNSUPPORTED_CACHES, cache


def rotary(**kw):
    r = B.SvRotary(P[30], None, None, 0, 64, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


BAD_ROTARY = [dict(freqs=None), dict(freqs=P[30] + 2), dict(dims=0), dict(dims=-16), dict(dims=80), dict(interleaved=2),
              dict(axes=P[31]), dict(ids=P[32], num_axes=0), dict(ids=P[32] + 1, num_axes=1),
              dict(ids=P[32], num_axes=2, axes=P[31] + 2)]
UNSUPPORTED_ROTARY = [dict(dims=8), dict(dims=24), dict(ids=P[32], num_axes=17)]
TOK, ROW = 6 * 64, 3 * 6 * 64       # q (2 heads), k (2) and values (2) of one projection, 3 tokens a row


def rotate(**kw):
    a = dict(q=P[0], q_row=ROW, q_tok=TOK, k=P[0] + 256, k_row=ROW, k_tok=TOK, rot=rotary(), positions=P[1], parents=None,
             lens=None, B=2, T=3, H=2, Hkv=2, D=64, qo=P[2], qo_row=3 * 128, qo_tok=128, ko=P[3], ko_row=3 * 128, ko_tok=128)
    a.update(kw)
    if a["rot"] is not None:
        a["rot"] = ctypes.byref(a["rot"])
    return B.load_library().spec_verify_rotate(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(rot=None), dict(positions=None), dict(B=0), dict(T=0),
    dict(H=0), dict(Hkv=0), dict(D=0), dict(q=P[0] + 8), dict(ko=P[3] + 2), dict(q_tok=TOK + 4), dict(k_row=-8),
    dict(qo_row=1 << 50),
    # outputs over themselves, each other, another's input, a part of their own, and lists
    dict(qo_tok=64), dict(qo_row=128), dict(ko=P[2]), dict(ko=P[2] + 128), dict(qo=P[0] + 256, qo_row=ROW, qo_tok=TOK),
    dict(ko=P[0], ko_row=ROW, ko_tok=TOK), dict(qo=P[0]), dict(qo=P[0] + 16, qo_row=ROW, qo_tok=TOK),
    dict(qo=P[0] + 512 + 144, qo_row=ROW, qo_tok=TOK), dict(qo=P[1] - 16), dict(ko=P[30]), dict(lens=P[2] + 4),
    dict(parents=P[3] + 8)])
def test_rotate_refuses(bad):
    assert rotate(**bad) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", BAD_ROTARY)
def test_rotate_refuses_bad_rotations(bad):
    assert rotate(rot=rotary(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", [dict(rot=rotary(**u)) for u in UNSUPPORTED_ROTARY] + [
    dict(D=72), dict(D=528), dict(T=65, parents=P[4], q_row=65 * TOK), dict(H=65537)])
def test_rotate_limits(bad):
    assert rotate(**bad) == B.SV_ERR_UNSUPPORTED


def append(**kw):
    a = dict(k=P[10], v=P[10] + 256, kv_row=3 * 256, kv_tok=256, T=3, lens=None, rot=rotary(), c=cache(), positions=P[13],
             blocks=P[14], positions_out=P[15], blocks_out=P[16], k_out=None, ko_row=0, ko_tok=0)
    a.update(kw)
    for k in ("c", "rot"):
        if a[k] is not None:
            a[k] = ctypes.byref(a[k])
    return B.load_library().spec_verify_append(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_append_refuses_bad_caches(bad):
    assert append(c=cache(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", UNSUPPORTED_CACHES)
def test_append_refuses_unsupported_caches(bad):
    assert append(c=cache(**bad)) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", BAD_ROTARY)
def test_append_refuses_bad_rotations(bad):
    assert append(rot=rotary(**bad)) == B.SV_ERR_ARG


K_OUT = dict(k_out=P[17], ko_row=3 * 128, ko_tok=128)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(positions=None), dict(blocks=None), dict(positions_out=None), dict(blocks_out=None),
    dict(T=0), dict(k=P[10] + 8), dict(kv_tok=4), dict(kv_row=-8), dict(kv_row=1 << 50), dict(positions_out=P[13]),
    dict(blocks_out=P[14]), dict(positions_out=P[16]), dict(positions_out=P[14]), dict(positions_out=P[13] + 4),
    dict(lens=P[15] + 4), dict(positions_out=P[6] + 8), dict(blocks_out=P[30]),
    dict(positions_out=P[10] + 16), dict(v=P[4]), dict(k=P[0]),                      # the prompt and what is written
    dict(K_OUT, k_out=P[17] + 8), dict(K_OUT, ko_tok=64), dict(K_OUT, ko_row=-8), dict(K_OUT, k_out=P[10] + 256),
    dict(k_out=P[10] + 256, ko_row=3 * 256, ko_tok=256), dict(k_out=P[10] + 16, ko_row=3 * 256, ko_tok=256),
    dict(K_OUT, k_out=P[4]), dict(K_OUT, k_out=P[15]), dict(K_OUT, k_out=P[13]), dict(K_OUT, lens=P[17] + 4)])
def test_append_refuses(bad):
    assert append(**bad) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", [dict(rot=rotary(**u)) for u in UNSUPPORTED_ROTARY] + [
    dict(T=(1 << 24) + 1), dict(T=1 << 24, c=cache(B=100, Hkv=64))])
def test_append_limits(bad):
    assert append(**bad) == B.SV_ERR_UNSUPPORTED


def test_gpu_tensors_only():
    with pytest.raises(ValueError):
        rsv.rotate_tokens(torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1, 64), torch.zeros(32))
    with pytest.raises(ValueError):
        rsv.cache_append(None, torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1, 64), None, None)
