"""cache_attention over shared prefixes, to the bits that spec_verify.h states
for a row's own pages: a probability beside a code has 11 bits, whatever the
value scales are.

Tolerance: that of tests/test_gpu_attention_range.py, for rows that have the
prefix's pages in their own tables, and what the join of prefix and row adds:
each enters with a weight from a base-2 logarithm or exponential of at most 2
smax + 32, off by 2^-23 of that at most, and up to 64 parts are added one after
the other, 2^-23 of the mean each.  Prefixes are multiples of 64 keys, so that
the tiles of both are the same.
"""

from __future__ import annotations

import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_attention import views
from tests.test_gpu_attention_range import bounds
from tests.test_gpu_prefix import run, shared_state

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
KINDS = ["e4m3", "int8"]


def state(seed, own, shared, starts, H, Hkv, D, page, kind, T, gain=1.0, near=1.0, q=1.0):
    """values of about `gain` in the pages and `near` in the tails and the new tokens."""
    s = shared_state(seed, own, shared, starts, Hkv=Hkv, D=D, page=page, kind=kind)
    rows, prefix, whole, before = s
    rows["v_scale"] *= gain             # the same tensor in both states
    for x in (rows, whole):
        x["v_tail"] = (x["v_tail"].float() * near).to(BF16)
    qkv = torch.randn((len(own), T, H + 2 * Hkv, D), generator=torch.Generator().manual_seed(seed + 1))
    qkv[:, :, :H] *= q
    qkv[:, :, H + Hkv:] *= near
    return s, qkv.to(BF16)


def check(s, qkv, H):
    rows, prefix, whole, before = s
    Hkv, D = rows["Hkv"], rows["D"]
    out, w = run(rows, prefix, qkv, H)
    ref, tol = bounds(whole, *views(qkv, H, Hkv), D ** -0.5)
    _, _, av, smax = R.attention(whole, *views(qkv, H, Hkv), D ** -0.5)
    tol += (2 * 2.0 ** -23 * (2 * smax + 32) + 64 * 2.0 ** -23)[..., None] * av * (1 + 2.0 ** -8)
    out = out.cpu().double()
    assert torch.isfinite(out).all()
    over = (out - ref).abs() / tol
    assert over.max() <= 1, (float(over.max()), float(((out - ref).abs() / ref.abs().amax()).max()))
    assert torch.equal(run(rows, prefix, qkv, H, weights=None).cpu().double(), out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D, page", [(64, 16), (128, 32), (64, 64), (128, 128)])
def test_probabilities_have_the_bits_of_a_rows_own(D, page, kind):
    """Two tokens of a prefix with opposite values, all others zero: what a probability loses stands alone."""
    s, qkv = state(1, [20, 5, 70, 0] * 4, [256 // page, 128 // page], [0, 9, 16], 8, 2, D, page, kind, 4, q=0.1)
    rows, prefix, whole, _ = s
    rows["v_pages"][:] = 0
    for i in range(2):
        p = int(prefix["prefix_table"][i, 0])
        one, less = (0x38, 0xB8) if kind == "e4m3" else (1, 0xFF)
        rows["v_pages"][p, :, :, 3], rows["v_pages"][p, :, :, 14] = one, less
    for x in (rows, whole):
        x["v_tail"].zero_()
    qkv[:, :, 10:] = 0
    check(s, qkv, 8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("e", [0, 6, -6, -20, -80, -100, 30, 100])
def test_values_of_every_magnitude(e, page, kind):
    gain = 2.0 ** e
    s, qkv = state(2, [100, 30, 0], [1280 // page, 128 // page], [0, 2, 3], 4, 2, 64, page, kind, 3, gain=gain, near=gain)
    check(s, qkv, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("gain, near", [(2.0 ** -10, 1.0), (1.0, 2.0 ** -20), (2.0 ** -60, 2.0 ** 50), (2.0 ** 60, 2.0 ** -60),
                                        (2.0 ** -100, 2.0 ** 120), (2.0 ** 100, 2.0 ** -100)])
def test_shared_values_unlike_the_rows(gain, near, page, kind):
    s, qkv = state(3, [100, 30, 0], [640 // page, 64 // page], [0, 2, 3], 4, 2, 128, page, kind, 3, near=near)
    p = s[1]["prefix_table"]
    s[0]["v_scale"][p[p >= 0].long()] *= gain
    check(s, qkv, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D, page", [(64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("span", [8, 40, 110])
def test_unlike_scales_in_one_part(span, D, page, kind):
    """Many heads, so that a work-group has many tiles of the prefix one after the other."""
    s, qkv = state(4, [3, page + 1], [2560 // page], [0, 2], 128, 128, D, page, kind, 1)
    g = torch.Generator().manual_seed(5)
    s[0]["v_scale"] *= torch.exp2(-span * torch.rand(s[0]["v_scale"].shape, generator=g) ** 2)
    check(s, qkv, 128)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D, page", [(64, 16), (128, 64)])
def test_zero_blocks_and_outliers_beside_small_values(D, page, kind):
    """A block of zeros has the scale 1; a channel of small values shows what its neighbours lose."""
    s, qkv = state(6, [3, 200], [2560 // page], [0, 2], 128, 128, D, page, kind, 1, gain=2.0 ** -30, near=2.0 ** -30)
    rows, prefix = s[:2]
    for j in range(1, 2560 // page, 3):
        p = int(prefix["prefix_table"][0, j])
        rows["v_pages"][p] = 0
        rows["v_scale"][p] = 1.0
        if j % 2:
            rows["v_pages"][p, :, 5] = 0x70 if kind == "e4m3" else 100
    check(s, qkv, 128)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("q", [3.0, 12.0])
def test_scores_far_apart(q, page, kind):
    """Tiles whose largest score lies far below the row's: their values still come with their bits in a channel
    where all others are zero."""
    s, qkv = state(7, [90, 0], [2560 // page], [0, 2], 128, 128, 64, page, kind, 1, q=q)
    rows, prefix, whole, _ = s
    per = max(1, 64 // page)
    for j in range(2560 // page):
        if j // per % 5:
            rows["v_pages"][int(prefix["prefix_table"][0, j]), :, 7] = 0
    for x in (rows, whole):
        x["v_tail"][..., 7] = 0
        for b in range(2):
            for j in range(int(rows["blocks"][b])):
                rows["v_pages"][int(rows["table"][b, j]), :, 7] = 0
    qkv[:, :, 256:, 7] = 0
    check(s, qkv, 128)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hkv, page", [(2, 16), (2, 64), (128, 64)])
def test_the_largest_and_smallest_values(Hkv, page, kind):
    """Means near the end of float32's range, of many parts and of one."""
    top = 2.0 ** (119 if kind == "e4m3" else 120)
    s, qkv = state(8, [0, 40, 0], [640 // page, 128 // page], [0, 2, 3], Hkv, Hkv, 64, page, kind, 2)
    rows, prefix = s[:2]
    p = prefix["prefix_table"]
    rows["v_pages"][p[0].long()] = 0x7E if kind == "e4m3" else 127     # 448 and 127: every mean is their value
    rows["v_scale"][p[0].long()] = top
    rows["v_scale"][p[1, :128 // page].long()] = 2.0 ** -126
    qkv[2, :, 2 * Hkv:] = 0
    check(s, qkv, Hkv)
