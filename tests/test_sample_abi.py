"""Argument checks of the calls that draw tokens and cut logits, on the host:
every call here returns before it launches anything."""

from __future__ import annotations

import ctypes

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_abi import P


def call(kind, ws=P[20], ws_n=None, **kw):
    a = dict(logits=P[0], row=3000, stride=1000, uniforms=P[1], T=P[2], k=P[3], p=P[4], m=P[5], B=2, P=3, V=1000, n=2,
             dtype=B.SV_BF16, tokens=P[6], logprobs=P[7], out=P[8], out_row=3000, out_stride=1000)
    a.update(kw)
    n = ctypes.c_size_t(1 << 40 if ws_n is None else ws_n)
    lib = B.load_library()
    if kind == "sample":
        rc = lib.spec_verify_sample(*(a[x] for x in ("logits", "row", "stride", "uniforms", "T", "k", "p", "m", "B", "P", "V",
                                                     "n", "dtype", "tokens", "logprobs")), ws, ctypes.byref(n), None)
    else:
        rc = lib.spec_verify_truncate(*(a[x] for x in ("logits", "row", "stride", "T", "k", "p", "m", "B", "P", "V", "dtype",
                                                       "out", "out_row", "out_stride")), ws, ctypes.byref(n), None)
    return rc if ws is not None else (rc, n.value)


BOTH = [dict(logits=None), dict(T=None), dict(B=0), dict(P=0), dict(V=0), dict(dtype=2), dict(stride=999), dict(row=2999),
        dict(stride=1 << 50, row=1 << 60), dict(logits=P[0] + 1), dict(T=P[2] + 2), dict(k=P[3] + 1), dict(p=P[4] + 2),
        dict(m=P[5] + 3), dict(ws=P[20] + 128), dict(ws=P[0] + 256), dict(ws=P[4] - 256)]


@pytest.mark.parametrize("bad", BOTH + [
    dict(uniforms=None), dict(tokens=None), dict(n=0), dict(uniforms=P[1] + 2), dict(tokens=P[6] + 1),
    dict(logprobs=P[7] + 2), dict(tokens=P[0] + 2), dict(tokens=P[1] + 44), dict(logprobs=P[6] + 44), dict(tokens=P[2] + 4),
    dict(logprobs=P[4]), dict(ws=P[6])])
def test_sample_refuses(bad):
    assert call("sample", **bad) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", BOTH + [
    dict(out=None), dict(out=P[8] + 1), dict(out_stride=999), dict(out_row=2999), dict(out=P[0], out_row=3001),
    dict(out=P[0] + 2), dict(out=P[0] - 11998), dict(out=P[2] + 4), dict(out=P[3] - 8), dict(ws=P[8] + 256)])
def test_truncate_refuses(bad):
    assert call("truncate", **bad) == B.SV_ERR_ARG


@pytest.mark.parametrize("kind", ["sample", "truncate"])
def test_limits_and_workspace(kind):
    big = (1 << 20) + 1
    assert call(kind, V=big, row=3 * big, stride=big) == B.SV_ERR_UNSUPPORTED
    assert call(kind, B=1 << 16, P=1 << 16, row=1 << 30) == B.SV_ERR_UNSUPPORTED
    assert call(kind, B=1 << 24, P=1) == B.SV_ERR_UNSUPPORTED
    rc, n = call(kind, ws=None)
    assert rc == B.SV_OK and n > 0 and n % 256 == 0
    assert call(kind, ws_n=n - 1) == B.SV_ERR_WORKSPACE
    rc, less = call(kind, ws=None, k=None, p=None, m=None)
    assert rc == B.SV_OK and less < n
    if kind == "sample":
        assert call(kind, n=B.SV_MAX_NODES + 1) == B.SV_ERR_UNSUPPORTED


def test_gpu_tensors_only():
    with pytest.raises(ValueError):
        rsv.sample_tokens(torch.zeros(1, 1, 8), torch.zeros(1, 1, 1), torch.ones(1))
    with pytest.raises(ValueError):
        rsv.truncate_logits(torch.zeros(1, 1, 8), torch.ones(1))
