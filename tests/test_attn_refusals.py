"""More host-side refusals of the attention layers' entry points (CPU: no kernel is launched)."""
import pytest

import gated_deltanet_speculative_gdn_gb300 as G
from test_attn_abi import dims, move, rope


# the cache of `dims()`: 8 pages of [16 tokens][2 heads][64]: 2048 elements a page, 16384 in all
@pytest.mark.parametrize("layers,stride", [
    (2, 0),             # every layer the same rows
    (2, 8), (3, 56),    # rows that overlap
    (2, 64),            # the next head of the same layer
    (2, 128),           # the next token
    (2, 2048),          # the next page
    (2, 16384 - 64),    # the last head of the last page
    (2, 1 << 39)])
def test_layers_that_share_rows_are_refused(layers, stride):
    assert move(dims(), layers=layers, ls=stride) == G.GDN_ERR_STRIDE


@pytest.mark.parametrize("layers,stride,kw", [
    # layers between the pages, the tokens and the heads, each with one layer more than there is room for
    (4, 2048, dict(page_stride=3 * 2048)), (4, 128, dict(token_stride=3 * 128, page_stride=16 * 3 * 128)),
    (4, 64, dict(head_stride=3 * 64, token_stride=6 * 64, page_stride=16 * 6 * 64))])
def test_layers_between_that_pass_into_the_next_are_refused(layers, stride, kw):
    assert move(dims(**kw), layers=layers, ls=stride) == G.GDN_ERR_STRIDE


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("columns", [-120, -8, 0, 8, 248])
def test_rows_of_one_buffer_that_share_columns_are_refused(name, columns):
    """q_out of 256 columns and k or v of 128 in rows of 1024: `columns` from q_out's first to the other's."""
    d = dims()
    at = 1 << 27
    assert rope(d, qo=at, qos=1024, **{name: at + 2 * columns, name + "s": 1024}) == G.GDN_ERR_ALIAS
    assert rope(d, qo=at, qos=1024, **{name: at + 2 * (columns + 1024), name + "s": 1024}) == G.GDN_ERR_ALIAS


def test_rows_of_two_strides_must_lie_apart():
    d = dims()
    at = 1 << 27
    assert rope(d, qo=at, qos=1024, k=at + 512, ks=512) == G.GDN_ERR_ALIAS
    assert rope(d, q=at, qs=1024, qo=at, qos=512) == rope(d, q=at, qs=1024, qo=at + 16, qos=1024) == G.GDN_ERR_ALIAS
