"""Arrays of the page calls that share memory are refused on the host, before
any device work (no GPU: the calls end at the missing tables)."""
import ctypes

import pytest

from decode_attention_dq_b200 import _native as N

NULL, SHAPE = -1, -4
P, MP, B_IN, B_OUT = 64, 8, 6, 5
WS = 1 << 20


def _sizes(op):
    rows, rows_out = (B_IN, B_OUT) if op == "fork" else (B_IN, B_IN)
    ins = dict(refs=P, table=rows * MP)
    outs = dict(refs_out=P, table_out=rows_out * MP)
    if op != "compact":
        ins.update(lens=rows, step=rows_out)
        outs.update(lens_out=rows_out)
    if op != "advance":
        outs.update(pairs=2 * (rows_out if op == "fork" else P // 2))
    outs.update(counts=8)
    return ins, outs


def _call(op, at):
    lib, p = N.load(), {k: ctypes.c_void_p(v) for k, v in at.items()}
    if op == "advance":
        return lib.dq_pages_advance(None, P, p["refs"], p["table"], MP, p["lens"], p["step"], B_IN, 0, 0, p["refs_out"],
                                    p["table_out"], p["lens_out"], p["counts"], p["ws"], WS, None)
    if op == "fork":
        return lib.dq_pages_fork(None, P, p["refs"], p["table"], MP, p["lens"], B_IN, p["step"], B_OUT, p["refs_out"],
                                 p["table_out"], p["lens_out"], p["pairs"], p["counts"], p["ws"], WS, None)
    return lib.dq_pages_compact(None, P, p["refs"], p["table"], MP, B_IN, p["refs_out"], p["table_out"], p["pairs"],
                                p["counts"], p["ws"], WS, None)


def _apart(op):
    """Addresses of arrays that lie one behind the other, without a gap."""
    ins, outs = _sizes(op)
    at, here = {}, 1 << 30
    for k, n in {**ins, **outs}.items():
        at[k] = here
        here += 4 * n
    at["ws"] = -(-here // 16) * 16
    return at


def _pairs(op):
    ins, outs = _sizes(op)
    names = list(outs) + ["ws"]
    return [(o, i) for o in names for i in list(ins) + names if o != i]


OPS = ("advance", "fork", "compact")


@pytest.mark.parametrize("op", OPS)
def test_neighbours_are_not_refused(op):
    assert _call(op, _apart(op)) == NULL


@pytest.mark.parametrize("op", OPS)
def test_an_output_that_is_another_array(op):
    own = {("refs_out", "refs"), ("table_out", "table"), ("lens_out", "lens"), ("lens_out", "step")}
    for out, other in _pairs(op):
        at = _apart(op)
        at[out] = at[other]
        assert _call(op, at) == (NULL if op != "fork" and (out, other) in own else SHAPE), (out, other)


@pytest.mark.parametrize("op", OPS)
def test_an_output_that_shares_some_of_another_array(op):
    ins, outs = _sizes(op)
    size = {**ins, **outs}
    for out, other in _pairs(op):
        if out == "ws":
            continue
        for start in (at_second, at_last) if other != "ws" else (at_second,):
            at = _apart(op)
            at[out] = start(at, out, other, size)
            assert _call(op, at) == SHAPE, (out, other, start.__name__)


def at_second(at, out, other, size):
    return at[other] + 4


def at_last(at, out, other, size):
    return at[other] - 4 * size[out] + 4
