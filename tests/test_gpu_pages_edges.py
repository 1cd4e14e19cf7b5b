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


def _fork(tab, refs, table, lens, parent):
    ins = [torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda() for x in (refs, table, lens, parent)]
    B, mp = table.shape
    n = len(parent)
    outs = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((len(refs),), (n, mp), (n,), (n, 2))]
    counts = dq.new_page_counts()
    ws = torch.empty(dq.dq_pages_workspace_bytes(tab, len(refs), max(B, n), mp), dtype=torch.uint8, device="cuda")
    dq.dq_pages_fork(tab, *ins, *outs, counts, ws)
    return (*outs, counts)


def test_forked_rows_do_not_share_what_they_will_write(tab):
    # Row 0 has taken tokens back: 40 are left, page 6 holds none of them. Row 1 ends with a block, page 3 lies past it
    # and is held by somebody else too. Row 2's page past its length is its own and it has one child.
    refs = np.array([1, 1, 1, 2, 0, 1, 1, 0, 1, 1])
    table = np.array([[0, 5, 6, -1], [1, 3, -1, -1], [2, 8, -1, 9]])
    got = _fork(tab, refs, table, [40, 32, 33], [0, 0, 1, 1, 2])
    _same(got, ([2, 2, 1, 1, 1, 1, 1, 0, 1, 1],
                [[0, 5, 6, -1], [0, 4, -1, -1], [1, -1, -1, -1], [1, -1, -1, -1], [2, 8, -1, 9]],
                [40, 40, 32, 32, 33], [(5, 4)] + [(-1, -1)] * 4, _counts(free_pages=1, taken=1, pairs=1)), "past the length")
    # Both children of row 0 go on: each in pages of its own.
    refs2, table2 = got[0].cpu().numpy(), got[1].cpu().numpy()[:2]
    grown = _advance(tab, np.r_[refs2, [0, 0]], table2, [40, 40], [30, 30])[1].tolist()
    assert grown == [[0, 5, 6, -1], [0, 4, 7, -1]]


def test_forks_of_long_rows_past_their_length(tab):
    # Rows of several segments of the kernel's, shortened inside each of them; one child, two, none.
    rng = np.random.default_rng(12)
    P, B, mp = 20000, 12, 1300
    refs, table, lens = R.random_state(rng, P, B, mp, share=0.0)
    cut = np.array([int(rng.integers(0, L + 1)) for L in lens])
    cut[3] = cut[3] // 32 * 32
    parent = [0, 1, 1, 3, 3, 4, 5, 5, 5, 7, 8, -1, 9, 9]
    got_refs, got_table, got_lens, _, got_counts = (x.cpu().numpy() for x in _fork(tab, refs, table, cut, parent))
    foreign = refs - np.bincount(table[table >= 0], minlength=P)
    assert np.array_equal(got_refs, foreign + np.bincount(got_table[got_table >= 0], minlength=P))
    seen = set()
    for c, p in enumerate(parent):
        if p < 0:
            assert (got_table[c] == -1).all()
            continue
        full = cut[p] // 32
        assert got_lens[c] == cut[p] and np.array_equal(got_table[c, :full], table[p, :full])
        if p not in seen:
            np.testing.assert_array_equal(got_table[c, full:], table[p, full:])
        else:
            last = full + (cut[p] % 32 > 0)
            assert (got_table[c, last:] == -1).all()
            assert (got_table[c, full:last] != table[p, full:last]).all()
        seen.add(p)
    own = [x for c, p in enumerate(parent) if p >= 0 for x in got_table[c, cut[p] // 32:] if x >= 0]
    assert len(own) == len(set(own)) and (got_refs[own] == 1).all()


def test_fork_counts_entries_out_of_range_once_per_child(tab):
    table = np.array([[0, 99, -1], [1, -7, 10], [2, 50, 3]])
    got = _fork(tab, np.array([1, 1, 1, 1]), table, [96, 96, 96], [0, 0, 1])
    _same(got, ([2, 1, 0, 0], [[0, -1, -1], [0, -1, -1], [1, -1, -1]], [96] * 3, [(-1, -1)] * 3,
                _counts(free_pages=2, bad=4)), "out of range")
