"""Argument checks of the operators around a verification round, on the host:
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
