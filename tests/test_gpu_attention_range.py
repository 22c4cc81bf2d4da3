"""cache_attention over the range of its values: value scales from 2^-126 to
2^119, unlike ones in one tile, rows whose mass lies far from their largest
score; to the bits that spec_verify.h states.

Tolerance, per output, with p the exact probabilities (their sum is 1), v the
values that the cache and the new tokens stand for, u = 2^-24:
 - scores are float32 sums of D exact products times two factors, so with S
   the largest sum of |scale q_d k_d| over the keys seen a score, and the
   argument of its exponential, is off by (D + 4) u S; with the denominator's
   the same, the exponentials' own 2 u, and sums of n terms (64 keys a tile,
   so at most n / 64 of them one after the other in each of two products, and
   16 a lane) in numerator and denominator:
     rel = 2 (D + 4) u S + 2^-20 + 2 u (n / 32 + 32);
 - p beside a code: 2^-11 of it, or of the largest p among the 64 cached keys
   of its tile 2^-21, 2^-16 where these are of several pages, whichever is more;
 - p beside the tail and the new tokens: 2^-16;
 - the output to bf16: 2^-8, and 2^-134 below bf16's normal range;
 - exponentials below 2^-100 of the largest may be lost (f16 follows the
   largest product no further): 2^-100 sum |v|; sums stay below 2^100, so
   what is 2^-120 of the largest sum may be lost: 2^-100 max over channels of
   sum p |v|; and a mean is formed in float32 times up to 2^-18: 2^-106.
"""

from __future__ import annotations

import pytest
import torch

import rejection_sampling_verifier_amd as rsv
from tests import cache_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
KINDS = ["e4m3", "int8"]


def bounds(s, q, kn, vn, scale, parents=None):
    """(out, tolerance) in float64."""
    B, T, H, D = q.shape
    Hkv, page, G = s["Hkv"], s["page"], H // s["Hkv"]
    u = 2.0 ** -24
    out, tol = (torch.zeros((B, T, H, D), dtype=torch.float64) for _ in range(2))
    for b in range(B):
        tail = R.tail_slots(s, b, s["k_tail"].shape[1])
        at = s["table"][b, :int(s["blocks"][b])].long()
        for h in range(Hkv):
            k = R.decode(s["k_pages"][at, h], s["kind"]) * s["k_scale"][at, h].double()[:, None, None]
            v = (R.decode(s["v_pages"][at, h], s["kind"]) * s["v_scale"][at, h].double()[:, None, None]).transpose(1, 2)
            k = torch.cat([k.reshape(-1, D), s["k_tail"][b, tail, h].double()])
            v = torch.cat([v.reshape(-1, D), s["v_tail"][b, tail, h].double()])
            nc = at.numel() * page
            for t in range(T):
                see = R.visible(None if parents is None else parents[b], T, t)
                kk, vv = torch.cat([k, kn[b, see, h].double()]), torch.cat([v, vn[b, see, h].double()])
                qq = q[b, t, h * G:(h + 1) * G].double()
                p = torch.softmax(qq @ kk.T * scale, 1)
                S = (qq.abs() @ kk.abs().T * scale).amax(1, keepdim=True)
                n = kk.shape[0]
                rel = 2 * (D + 4) * u * S + 2.0 ** -20 + 2 * u * (n / 32 + 32)
                ref = p @ vv
                err = rel * (p @ vv.abs()) + 2.0 ** -16 * (p[:, nc:] @ vv[nc:].abs())
                tiles = torch.nn.functional.pad(p[:, :nc], (0, -nc % 64)).reshape(G, -1, 64)
                least = (2.0 ** (-21 if page >= 64 else -16) * tiles.amax(2, keepdim=True)).expand_as(tiles)
                err += torch.maximum(2.0 ** -11 * p[:, :nc], least.reshape(G, -1)[:, :nc]) @ vv[:nc].abs()
                err += 2.0 ** -100 * (vv.abs().sum(0) + (p @ vv.abs()).amax(1, keepdim=True)) + 2.0 ** -106
                out[b, t, h * G:(h + 1) * G] = ref
                tol[b, t, h * G:(h + 1) * G] = err + 2.0 ** -8 * (ref.abs() + err) + 2.0 ** -134
    return out, tol


def check(s, qkv, H, parents=None, weights=True):
    Hkv, D = s["Hkv"], s["D"]
    part = lambda x: (x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:])  # noqa: E731
    cache, positions, blocks = R.to_gpu(s)
    got = rsv.cache_attention(*part(qkv.cuda()), cache, positions, blocks, weights=weights,
                              parents=None if parents is None else parents.cuda())
    ref, tol = bounds(s, *part(qkv), D ** -0.5, parents)
    out = (got[0] if weights else got).cpu().double()
    assert torch.isfinite(out).all()
    over = (out - ref).abs() / tol
    assert over.max() <= 1, (float(over.max()), float(((out - ref).abs() / ref.abs().amax()).max()))
    if weights:
        _, w, _, smax = R.attention(s, *part(qkv), D ** -0.5, parents)
        r = 2 * (D + 4) * 2.0 ** -24 * smax.amax(2) + 2.0 ** -20 + 4 * 2.0 ** -23 * (smax.amax(2) + 32)
        r += 2.0 ** -23 * (s["table"].shape[1] * s["page"] / 32 + 32)
        assert ((got[1].cpu().double() - w).abs() <= r[..., None] * w + 1e-30).all()


def state(seed, contexts, H, Hkv, D, page, kind, T, gain=1.0, strong=0.0, near=1.0):
    """values of about `gain` in the cache and `near` in the tail and the new tokens; strong: how far the newest
    token's score lies over the others' (in powers of two)."""
    B = len(contexts)
    s = R.random_state(seed, B=B, Hkv=Hkv, D=D, page=page, kind=kind, contexts=contexts)
    s["v_scale"] *= gain
    s["v_tail"] = (s["v_tail"].float() * near).to(BF16)
    g = torch.Generator().manual_seed(seed + 1)
    qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g)
    if strong:
        G = H // Hkv
        base = torch.randn((B, T, Hkv, 1, D), generator=g)
        qkv[:, :, :H] = (base + 0.1 * torch.randn((B, T, Hkv, G, D), generator=g)).reshape(B, T, H, D)
        unit = base[:, :, :, 0] / base[:, :, :, 0].norm(dim=-1, keepdim=True) ** 2
        qkv[:, :, H:H + Hkv] = unit * (strong * 0.6931 * D ** 0.5)
    qkv[:, :, H + Hkv:] *= near
    return s, qkv.to(BF16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("e", [6, -6, -12, -20, -40, -80, -100, 30, 100])
def test_values_of_every_magnitude(e, page, kind):
    gain = 2.0 ** e
    s, qkv = state(1, [2500, 130, 0, 700], 4, 2, 64, page, kind, 3, gain=gain, near=gain)
    check(s, qkv, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gain, near", [(2.0 ** -10, 1.0), (1.0, 2.0 ** -20), (2.0 ** -60, 2.0 ** 50),
                                        (2.0 ** 60, 2.0 ** -60), (2.0 ** -100, 2.0 ** 120), (2.0 ** 100, 2.0 ** -100)])
def test_cached_values_unlike_the_new_ones(gain, near, kind):
    s, qkv = state(2, [2500, 130, 64, 700], 4, 2, 128, 32, kind, 3, gain=gain, near=near)
    check(s, qkv, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D, page", [(64, 64), (128, 16)])
@pytest.mark.parametrize("strong", [6.0, 10.0, 14.0, 20.0])
def test_a_strong_new_token_before_small_values(strong, D, page, kind):
    """Long rows over many heads, so that the wave which meets the new token also takes many cached tiles."""
    s, qkv = state(3, [16384 + 40, 9000], 8, 8, D, page, kind, 1, gain=2.0 ** -12, near=2.0 ** -12, strong=strong)
    check(s, qkv, 8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D, page", [(64, 64), (128, 16)])
@pytest.mark.parametrize("gain, near", [(2.0 ** -100, 2.0 ** 120), (2.0 ** -60, 2.0 ** 100), (2.0 ** -110, 1.0),
                                        (2.0 ** 100, 2.0 ** -100), (2.0 ** -20, 2.0 ** 20)])
def test_ends_of_the_range_in_one_wave(gain, near, D, page, kind):
    """Rows as long as above: what a wave's sums cannot hold beside each other still counts in the denominator."""
    s, qkv = state(10, [16384 + 40, 9000], 8, 8, D, page, kind, 1, gain=gain, near=near)
    check(s, qkv, 8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("span", [8, 40, 110])
def test_unlike_scales_in_one_wave(span, page, kind):
    s, qkv = state(4, [6000, 200, 3000], 8, 4, 64, page, kind, 2)
    g = torch.Generator().manual_seed(5)
    s["v_scale"] *= torch.exp2(-span * torch.rand(s["v_scale"].shape, generator=g) ** 2)
    check(s, qkv, 8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H, D, page", [(8, 64, 16), (16, 128, 32), (64, 64, 16), (8, 128, 64)])
def test_zero_blocks_and_outliers_beside_small_values(H, D, page, kind):
    """A block of zeros has the scale 1; a channel of small values shows what its neighbours lose."""
    s, qkv = state(6, [12000, 150, 5900], H, 8, D, page, kind, 4 if H > 8 else 1, gain=2.0 ** -30, near=2.0 ** -30)
    for b in range(3):
        for j in range(1, int(s["blocks"][b]), 3):
            p = int(s["table"][b, j])
            s["v_pages"][p] = 0
            s["v_scale"][p] = 1.0
            if j % 2:
                s["v_pages"][p, :, 5] = 0x70 if kind == "e4m3" else 100
    check(s, qkv, H)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gain", [3.0, 12.0])
def test_scores_far_apart(gain, kind):
    """Tiles whose largest score lies far below the row's: their values still come with their bits in a channel
    where all others are zero."""
    s, qkv = state(7, [4000, 90, 1500], 4, 2, 64, 64, kind, 2)
    qkv[:, :, :4] = (qkv[:, :, :4].float() * gain).to(BF16)
    s["v_tail"][..., 7] = 0
    qkv[:, :, 6:, 7] = 0
    for b in range(3):
        for j in range(int(s["blocks"][b])):
            if j % 5:
                s["v_pages"][int(s["table"][b, j]), :, 7] = 0
    check(s, qkv, 4)


def test_trees_and_many_queries_to_a_head():
    for kind in KINDS:
        for D in (64, 128):
            s, qkv = state(8, [3000, 70], 16, 2, D, 64, kind, 13, gain=2.0 ** -14, near=2.0 ** -14, strong=9.0)
            par = torch.zeros((2, 13), dtype=torch.int32)
            par[:, 1:] = torch.arange(12) // 2
            check(s, qkv, 16, parents=par)


@pytest.mark.parametrize("kind", KINDS)
def test_the_largest_and_smallest_values(kind):
    """One visible token of bf16's largest value, and blocks at the ends of float32's range of scales."""
    s, qkv = state(9, [0, 40, 64, 128], 2, 2, 64, 16, kind, 2)
    qkv[0, :, 4:] = torch.finfo(BF16).max
    s["v_scale"][s["table"][1, :2].long()] = 2.0 ** -126
    qkv[1, :, 4:], s["v_tail"][1] = 0.0, 0.0
    top = 2.0 ** (119 if kind == "e4m3" else 120)
    s["v_scale"][s["table"][2, :4].long()] = top
    s["v_scale"][s["table"][3, :4].long()] = 2.0 ** -126
    s["v_scale"][s["table"][3, 4:8].long()] = top
    check(s, qkv, 2)
