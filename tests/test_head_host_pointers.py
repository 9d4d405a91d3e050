"""Pointers that are not aligned to their type are refused on the host (a kernel that read them
would fault), and so are outputs that other rows are still read from. Without a GPU; no pointer is
dereferenced."""

import pytest

from tests.test_head_host import BF16, E4M3, F32, FAKE, SHAPE, WORKSPACE, _norm, _process, _project, lib  # noqa: F401 (a fixture)

LISTS = dict(off=FAKE, B=4, hist=FAKE, hoff=FAKE, total=40, prompt=FAKE, rep=FAKE, freq=FAKE, pres=FAKE, bt=FAKE, bv=FAKE,
             bo=FAKE, nb=10, mask=FAKE, mi=FAKE)


@pytest.mark.parametrize("name", ["off", "hist", "hoff", "prompt", "rep", "freq", "pres", "bt", "bv", "bo", "mask", "mi"])
def test_process_refuses_unaligned_lists(lib, name):  # noqa: F811
    for by in (1, 2, 3):
        assert _process(lib, **dict(LISTS, **{name: FAKE + by})) == SHAPE


@pytest.mark.parametrize("name", ["scale", "ids", "off"])
def test_project_refuses_unaligned_lists(lib, name):  # noqa: F811
    adapters = dict(la=FAKE, lb=FAKE, A=2, rank=8, ids=FAKE, scale=FAKE, off=FAKE, B=4)
    for by in (1, 2, 3):
        assert _project(lib, **dict(adapters, **{name: FAKE + by})) == SHAPE


def test_clear_status_refuses_what_is_no_workspace(lib):  # noqa: F811
    assert lib.lp_head_clear_status(FAKE + 4, None) == WORKSPACE


def test_norm_refuses_what_cannot_be_done_in_place(lib):  # noqa: F811
    other, more = 2 * FAKE, 3 * FAKE
    picked = dict(rows=4 * FAKE, n=2, ws=FAKE, wsb=256)
    # picked rows: a row may be read after another one has been written over it
    assert _norm(lib, x=other, out=other, **picked) == SHAPE
    assert _norm(lib, x=other, residual=more, out=more, **picked) == SHAPE
    assert _norm(lib, x=other, kept=other, **picked) == SHAPE
    assert _norm(lib, x=other, residual=more, kept=more, **picked) == SHAPE
    # another type or stride
    assert _norm(lib, x=other, out=other, odtype=F32) == SHAPE
    assert _norm(lib, x=other, out=other, odtype=E4M3, scale=more) == SHAPE
    assert _norm(lib, x=other, out=other, os_=72) == SHAPE and _norm(lib, x=other, kept=other, ks=72) == SHAPE
    assert _norm(lib, x=other, out=more, kept=more) == SHAPE                # two outputs in one place


def test_no_rows_is_a_size_and_not_a_missing_pointer(lib):  # noqa: F811
    assert _norm(lib, x=None, out=None, T=0, n=0) == SHAPE and _norm(lib, out=None, rows=FAKE, n=0, ws=FAKE, wsb=256) == SHAPE
    assert _project(lib, x=None, out=None, T=0) == SHAPE and _project(lib, w=None, out=None, V=0) == SHAPE
    assert _process(lib, x=None, out=None, T=0, B=0) == SHAPE
    assert "aligned" in lib.lp_ragged_strerror(SHAPE).decode() and "stride" in lib.lp_ragged_strerror(SHAPE).decode()
