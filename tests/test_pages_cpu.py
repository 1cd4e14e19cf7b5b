"""Refusals of the page calls (no GPU) and properties of their definitions."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import decode_attention_dq_b200 as dq
from decode_attention_dq_b200 import _native as N
from tests import _pages as R

NULL, SHAPE, ALIGN = -1, -4, -6
P4, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4098)


def test_count_fields_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dq.h")).read()
    body = re.sub(r"/\*.*?\*/", "", re.search(r"typedef struct \{([^}]*)\} dq_page_counts;", text, flags=re.S).group(1), flags=re.S)
    assert tuple(re.findall(r"int32_t (\w+);", body)) == N.PAGE_COUNT_FIELDS


def test_argument_errors_come_before_any_device_work():
    lib = N.load()
    assert lib.dq_pages_workspace_bytes(None, 8, 1, 4) == 0
    assert lib.dq_pages_advance(None, 8, None, None, 4, None, None, 1, 0, 0, None, None, None, None, None, 0, None) == NULL
    assert lib.dq_pages_advance(None, 8, P4, P4, 4, P4, P4, 1, -1, 0, P4, P4, P4, P4, P4, 0, None) == SHAPE
    assert lib.dq_pages_advance(None, 8, P4, P4, 4, P4, P4, 1, 0, -1, P4, P4, P4, P4, P4, 0, None) == SHAPE
    assert lib.dq_pages_advance(None, 8, P4, P4, 4, ODD, P4, 1, 0, 0, P4, P4, P4, P4, P4, 0, None) == ALIGN
    assert lib.dq_pages_fork(None, 8, P4, P4, 4, P4, 1, P4, 1, P4, P4, P4, P4, P4, P4, 0, None) == SHAPE  # outputs are inputs
    assert lib.dq_pages_fork(None, 8, None, None, 4, None, 1, None, 1, None, None, None, None, None, None, 0, None) == NULL
    assert lib.dq_pages_compact(None, 8, None, None, 4, 1, None, None, None, None, None, 0, None) == NULL
    assert lib.dq_pages_compact(None, 8, P4, P4, 4, 1, P4, P4, ODD, P4, P4, 0, None) == ALIGN
    assert lib.dq_pages_copy(None, P4, P4, 8, 1, 0, 0, P4, 1, None, None, None) == NULL


def test_binding_refuses_tensors_that_do_not_fit():
    r, t, L = dq.new_page_state(8, 2, 4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        dq.dq_pages_advance(None, r, t, L, L, r, t, L, r, r)
    with pytest.raises(ValueError, match="refs"):
        N._check_int32("lens refs", (L, (2,)), (r, (9,)))
    with pytest.raises(ValueError, match="lens"):
        N._check_int32("lens", (L.long(), (2,)))


@pytest.mark.parametrize("seed", range(6))
def test_definitions_keep_the_references_whole(seed):
    """After every call each page has as many references as table entries name it, plus those that no row held."""
    rng = np.random.default_rng(seed)
    P, B, mp, window = 90, 7, 12, int(rng.choice([0, 60]))
    refs, table, lens = R.random_state(rng, P, B, mp, window=window)
    foreign = refs - np.bincount(table[table >= 0], minlength=P)
    assert (foreign >= 0).all()

    def whole():
        return np.array_equal(np.array(refs), foreign + np.bincount(table[table >= 0], minlength=P))

    for _ in range(12):
        refs, table, lens, c = R.advance(refs, table, lens, rng.choice([-1, 1, 1, 40], len(lens)), window)
        assert whole() and c["free_pages"] == sum(v == 0 for v in refs)
        refs, table, lens, pairs, c = R.fork(refs, table, lens, rng.integers(-1, len(lens), B))
        assert whole()
        for b, L in enumerate(lens):  # a partly filled last page is nobody else's
            if L % 32 and table[b, L // 32] >= 0 and foreign[table[b, L // 32]] == 0:
                assert refs[table[b, L // 32]] == 1
        refs, table, pairs, c = R.compact(refs, table)
        for s, d in pairs[:c["pairs"]]:
            foreign[d], foreign[s] = foreign[s], 0
        assert whole()
        live = P - c["free_pages"]
        assert all(v > 0 for v in refs[:live]) and not any(refs[live:])
