"""Calls at the edges of the page calls' contract (dq.h), each against values
written out here or against the definition of tests/_pages.py."""
import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from tests import _common as cm
from tests import _pages as R
from tests.test_gpu_pages import _advance, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tab():
    return cm.lib_tables(2)


def _counts(**named):
    return dict.fromkeys(dq._native.PAGE_COUNT_FIELDS, 0) | named


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("window", [0, 33])
def test_a_row_without_new_tokens_takes_no_page(tab, window, in_place):
    # Length 40 with the page of tokens 32 .. 39 missing (an earlier call ran short): no new token, no page. The next
    # row is whole, the last one's page is missing too and its new token 40 takes the lowest free one.
    refs = np.array([1, 0, 0, 1, 1, 1])
    table = np.array([[5, -1, -1], [4, 3, -1], [0, -1, -1]])
    got = _advance(tab, refs, table, [40, 40, 40], [0, 0, 1], window, 0, in_place)
    left = [-1 if window == 1 else 0, 1, -1]
    _same(got, ([1, 1, 0, 1, 1, 1], [[5, -1, -1], [4, 3, -1], left], [40, 40, 41], _counts(free_pages=1, taken=1)), "n = 0")


def test_rows_without_new_tokens_in_a_large_state(tab):
    # Above the size of one launch.
    P, B, mp = 660001, 30, 701
    rng = np.random.default_rng(6)
    refs, table, lens = R.random_state(rng, P, B, mp)
    lens = lens // 32 * 32 - 15  # every row ends inside a block
    lens[lens < 0] = 20
    for b, L in enumerate(lens):
        p = table[b, L // 32]
        if b % 3 == 0 and p >= 0:
            refs[p] -= 1
            table[b, L // 32] = -1
    n = np.where(np.arange(B) % 2 == 0, 0, 40)
    got = _advance(tab, refs, table, lens, n)
    still = got[1].cpu().numpy()
    assert np.array_equal(still[::2], table[::2]) and (table[::6, :].min(1) == -1).all()
    want = R.advance(refs, table[1::2], lens[1::2], n[1::2])
    np.testing.assert_array_equal(still[1::2], want[1])
    np.testing.assert_array_equal(got[0].cpu().numpy(), want[0])
    assert dq.page_counts_dict(got[3]) == want[3]


def test_a_full_row_takes_no_page(tab):
    # The row is as long as the table allows: new tokens are clamped, nothing is wanted.
    got = _advance(tab, np.array([1, 0, 0]), np.array([[0, -1]]), [64], [7])
    _same(got, ([1, 0, 0], [[0, -1]], [64], _counts(free_pages=2, clamped=1)), "full")
