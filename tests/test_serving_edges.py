"""Argument checks of the operators around a verification step that lie at the
edges of what they take, on the host: every call here returns before it
launches anything."""

from __future__ import annotations

import pytest

import rejection_sampling_verifier_amd as rsv
from rejection_sampling_verifier_amd import binding as B
from tests.test_serving_resources import kernels  # noqa: F401
from tests.test_serving_abi import OUT, P, WEIGHTS, adjust, attention, cache, commit, evict


@pytest.mark.parametrize("width", [-1, 5])
def test_a_history_is_no_wider_than_its_rows_are_apart(width):
    assert adjust(c_repetition=P[3], c_history=P[5], c_history_lens=P[6], c_history_stride=4,
                  c_history_width=width) == B.SV_ERR_ARG


COUNTERS, TOTALS, NODES = 2 * 4, 2 * 10 * 4, 4 * (5 + 2)


@pytest.mark.parametrize("bad", [
    dict(totals_out=P[19]), dict(totals_out=P[19] + WEIGHTS - 4), dict(totals_out=P[19] + 4 - TOTALS),   # over weights
    dict(totals_out=P[6]), dict(totals_out=P[12] + 4), dict(totals_out=P[13]), dict(totals_out=P[14] + 4 - TOTALS),
    dict(totals_out=P[17] + NODES - 4), dict(totals_out=P[15]), dict(totals_out=P[16] - TOTALS + 4),
    dict(positions_out=P[6] + TOTALS - 4), dict(blocks_out=P[17] + NODES - 4), dict(positions_out=P[19]),
    dict(blocks_out=P[18] + 4)])
def test_commit_refuses_outputs_over_what_it_reads(bad):
    a = dict(nodes=P[17], stride=5, weights=P[19], totals=P[18], totals_out=P[20])
    assert commit(**dict(a, **bad)) == B.SV_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(evicted=P[0]), dict(evicted=P[1] + 1600 - 4), dict(evicted=P[3] + 8), dict(evicted=P[4] - 12),
    dict(blocks_out=P[0] + 1596), dict(blocks_out=P[1]), dict(blocks_out=P[3] - 12), dict(blocks_out=P[4]),
    dict(totals_out=P[2] - 1596), dict(table_out=P[2])])
def test_evict_refuses_outputs_over_what_it_reads(bad):
    assert evict(**bad) == B.SV_ERR_ARG


PAGES, TAIL = 100 * 2 * 16 * 64, 2 * 32 * 2 * 64 * 2


@pytest.mark.parametrize("bad", [
    dict(out=P[20]), dict(out=P[20] + 16 - OUT), dict(weights=P[20] + 64), dict(weights=P[0] + PAGES - 4),
    dict(out=P[1]), dict(out=P[4] + TAIL - 16), dict(weights=P[5]), dict(weights=P[2] + 796), dict(out=P[3]),
    dict(out=P[6]), dict(weights=P[13] + 4), dict(weights=P[14] + 4 - WEIGHTS), dict(out=P[16], parents=P[16]),
    dict(weights=P[17], lens=P[17])])
def test_attention_refuses_outputs_over_any_input(bad):
    assert attention(**bad) == B.SV_ERR_ARG


def test_launches_of_2_to_the_32_work_items_are_refused():
    """A launch counts its work-items in 32 bits."""
    far = P[0] + (1 << 50)
    one = dict(P=1, V=4096, row=4096, stride=4096, out_row=4096, out_stride=4096, out=far)
    assert adjust(B=2 ** 24, **one) == B.SV_ERR_UNSUPPORTED
    biased = dict(one, c_bias_ids=P[7], c_bias_values=P[8], c_bias_stride=2049)
    assert adjust(B=2 ** 23, **biased) == B.SV_ERR_UNSUPPORTED
    big = cache(B=65536, Hkv=128, num_pages=1, max_blocks=1)
    for i, k in enumerate(("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail", "block_table")):
        setattr(big, k, (1 << 50) + (i << 44))
    assert commit(c=big, kn=1 << 52, vn=1 << 53) == B.SV_ERR_UNSUPPORTED
    many = cache(B=65536, Hkv=1, max_blocks=65536, page=16)
    assert attention(c=many, H=1, T=1, weights=P[16], ws=None)[0] == B.SV_ERR_UNSUPPORTED
    assert evict(B=2 ** 22, most=1, totals=1 << 50, table=1 << 51, totals_out=1 << 52, table_out=1 << 53,
                 blocks=1 << 54, blocks_out=1 << 55, evicted=1 << 56) == B.SV_ERR_UNSUPPORTED


def test_rows_of_more_tiles_than_32_bits_count_are_refused():
    """8191 rows of 65536 blocks of 256 tokens are nearly 2^31 tiles, which a rounded-up division carries past it."""
    for b, hkv in ((8191, 1), (4097, 1024)):
        assert attention(c=cache(B=b, Hkv=hkv, page=256, max_blocks=65536, tail=512), H=hkv, T=1,
                         ws=None)[0] == B.SV_ERR_UNSUPPORTED
    assert attention(c=cache(B=2000, Hkv=1, page=256, max_blocks=65536, tail=512), H=1, T=1, ws=None)[0] == B.SV_OK


def test_rows_of_2_to_the_30_entries_are_refused():
    """A count shares its word with two flags, and indices run past a row's end by a work-group's stride."""
    n = 2 ** 30
    hist = dict(c_repetition=P[3], c_history=P[5], c_history_lens=P[6])
    assert adjust(c_history_stride=n, **hist) == B.SV_ERR_UNSUPPORTED
    assert adjust(c_history_stride=2 * n - 1, c_history_width=n, **hist) == B.SV_ERR_UNSUPPORTED
    assert adjust(c_bias_ids=P[7], c_bias_values=P[8], c_bias_stride=2 * n - 2) == B.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(B=0), dict(num_pages=0), dict(Hkv=0), dict(D=0), dict(page=0), dict(max_new=0),
                                 dict(max_blocks=0), dict(B=-1)])
def test_new_cache_refuses_empty_sizes(bad):
    with pytest.raises(ValueError):
        rsv.new_cache(**dict(dict(B=1, num_pages=4, Hkv=1, D=64, page=16), **bad))


def test_four_adjusting_work_groups_to_a_cu(kernels):  # noqa: F811
    mine = [v for k, v in kernels.items() if "adjust_logits_kernel" in k]
    assert len(mine) == 2
    for v in mine:
        assert int(v["Occupancy [waves/SIMD]"]) >= 4 and 4 * int(v["LDS Size [bytes/block]"]) <= 160 * 1024, v
