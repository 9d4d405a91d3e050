"""Pointers that are not aligned to their type are refused on the host: a kernel that read them
would fault. Without a GPU; no pointer is dereferenced."""

import pytest

from tests.test_head_host import FAKE, SHAPE, WORKSPACE, _process, _project, lib  # noqa: F401 (a fixture)

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
