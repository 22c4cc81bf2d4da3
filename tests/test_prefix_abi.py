"""Argument checks of attention over shared prefixes, on the host: every call
here returns before it launches anything."""

from __future__ import annotations

import ctypes

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_abi import BAD_CACHES, P, UNSUPPORTED_CACHES, cache


def prefix(**kw):
    p = B.SvPrefix(P[40], P[41], P[42], 3, 20)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def attention(ws=P[20], ws_n=None, **kw):
    a = dict(q=P[10], q_row=3 * 512, q_tok=512, kn=P[11], vn=P[12], kv_row=3 * 512, kv_tok=512, c=cache(), prefix=prefix(),
             positions=P[13], blocks=P[14], parents=None, lens=None, T=3, H=4, scale=0.125, out=P[15], weights=None)
    a.update(kw)
    n = ctypes.c_size_t(1 << 40 if ws_n is None else ws_n)
    for k in ("c", "prefix"):
        if a[k] is not None:
            a[k] = ctypes.byref(a[k])
    rc = B.load_library().spec_verify_attention_prefix(*a.values(), ws, ctypes.byref(n), None)
    return rc if ws is not None else (rc, n.value)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_refuses_bad_caches(bad):
    assert attention(c=cache(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", UNSUPPORTED_CACHES)
def test_refuses_unsupported_caches(bad):
    assert attention(c=cache(**bad)) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(table=None), dict(blocks=None), dict(starts=None), dict(count=0), dict(count=-1),
                                 dict(max_blocks=0), dict(table=P[40] + 2), dict(blocks=P[41] + 1), dict(starts=P[42] + 3),
                                 dict(table=P[15]), dict(blocks=P[15] + 8), dict(starts=P[15] - 8), dict(table=P[20] + 4096)])
def test_refuses_bad_prefixes(bad):
    assert attention(prefix=prefix(**bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", [dict(count=65537), dict(max_blocks=B.SV_MAX_BLOCKS + 1)])
def test_refuses_unsupported_prefixes(bad):
    assert attention(prefix=prefix(**bad)) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(T=0), dict(H=3), dict(scale=0.0), dict(out=P[10]),
                                 dict(ws=P[20] + 16), dict(weights=P[15])])
def test_refuses(bad):
    assert attention(**bad) == B.SV_ERR_ARG


def test_limits_and_workspace():
    assert attention(T=B.SV_MAX_K + 2) == B.SV_ERR_UNSUPPORTED
    big = cache(B=65536, Hkv=256)
    assert attention(c=big, prefix=prefix(count=65536), T=1, H=256, q_row=256 * 64, q_tok=256 * 64, kv_row=256 * 64,
                     kv_tok=256 * 64, out=P[15] + (1 << 50)) == B.SV_ERR_UNSUPPORTED
    rc, n = attention(ws=None)
    assert rc == B.SV_OK and n > 0 and n % 256 == 0
    rc, without = attention(ws=None, prefix=None)
    assert rc == B.SV_OK and without < n
    rc, more = attention(ws=None, prefix=prefix(max_blocks=2000))
    assert rc == B.SV_OK and more > n
    rc, heavy = attention(ws=None, weights=P[16])
    assert rc == B.SV_OK and heavy > n
    assert attention(ws_n=n - 1) == B.SV_ERR_WORKSPACE
