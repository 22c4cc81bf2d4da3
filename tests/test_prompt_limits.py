"""Launches of 2^32 work-items and more are refused before anything runs, on the
host: sizes at the border of what the calls that bring prompts in and draw
tokens take.  Every call here is a size query or is refused."""

from __future__ import annotations

import ctypes

import pytest

from rejection_sampling_verifier_amd import binding as B
from tests.test_prefix_abi import attention, prefix
from tests.test_sample_abi import call
from tests.test_serving_abi import P, cache


@pytest.mark.parametrize("dtype, part", [(B.SV_BF16, 8192), (B.SV_F32, 4096)])
def test_truncate_counts_the_work_groups_of_its_last_kernel(dtype, part):
    """It has one to `part` logits (and a lead of one vector), the first one to twice as many."""
    rows, V = 1 << 23, part + 1
    one = dict(P=1, V=V, row=V, stride=V, out_row=V, out_stride=V, dtype=dtype)
    rc, n = call("truncate", ws=None, B=rows - 1, **one)
    assert rc == B.SV_OK and n > 0
    rc, _ = call("truncate", ws=None, B=rows, **one)
    assert rc == B.SV_ERR_UNSUPPORTED
    assert call("truncate", B=rows, **dict(one, out=P[0])) == B.SV_ERR_UNSUPPORTED   # in place
    rc, n = call("sample", ws=None, B=rows, **{k: one[k] for k in ("P", "V", "row", "stride", "dtype")})
    assert rc == B.SV_OK and n > 0


@pytest.mark.parametrize("D, H", [(64, 64), (128, 32)])
def test_prefix_counts_the_work_groups_of_its_join(D, H):
    """D / 4 work-items to a token's head: B T H D below 2^34."""
    def rc(B_, H_):
        heads = dict(T=64, H=H_, q_row=64 * H_ * D, q_tok=H_ * D, kv_row=64 * H_ * D, kv_tok=H_ * D)
        return attention(ws=None, c=cache(B=B_, Hkv=H_, D=D, max_blocks=1), prefix=prefix(count=1, max_blocks=1), **heads)
    assert rc(65536, H)[0] == B.SV_ERR_UNSUPPORTED
    code, n = rc(65535, H)
    assert code == B.SV_OK and n > 0


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 26])
def test_rotate_counts_tokens_past_32_bits(T):
    rot = B.SvRotary(P[9], None, None, 0, 16, 0)
    n = 1 << 10
    rc = B.load_library().spec_verify_rotate(P[0] << 16, 0, n, P[1] << 16, 0, n, ctypes.byref(rot), P[5], None, None, 1, T, 1, 1,
                                             16, P[2] << 16, 0, n, P[3] << 16, 0, n, None)
    assert rc == B.SV_ERR_UNSUPPORTED
