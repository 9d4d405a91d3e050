"""Host checks of the head operators: the header's symbols, and every refusal, without a GPU
(each call returns before anything is enqueued; the pointers are never dereferenced)."""

import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
OK, NULL, SHAPE, WORKSPACE, DTYPE = 0, 1, 3, 6, 9
F32, BF16, F16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from ragged_log_probs_gb300 import _build
    _build.build()
    import ragged_log_probs_gb300 as lp
    return lp.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = open(os.path.join(ROOT, "include", "lp_head.h")).read()
    names = set(re.findall(r"^\s*(?:lp_status|size_t)\s+(lp_\w+)\s*\(", text, flags=re.M))
    assert names >= {"lp_head_workspace_size", "lp_head_clear_status", "lp_head_norm", "lp_head_project", "lp_head_process"}
    for name in names:
        assert getattr(lib, name).argtypes, name


def test_new_error_codes_have_texts(lib):
    texts = {lib.lp_ragged_strerror(c).decode() for c in range(13)}
    assert len(texts) == 13 and "unknown lp_status" not in texts


def test_workspace_size(lib):
    assert lib.lp_head_workspace_size(0, 0) == 256
    assert lib.lp_head_workspace_size(10, 0) == 256
    # header, a page and factors of 256 rows, u padded to 16 columns, its parts in 64
    assert lib.lp_head_workspace_size(10, 8) == 256 + 2560 + 256 * (4 + 64 + 128)
    assert lib.lp_head_workspace_size(1, 65) == 0
    assert lib.lp_head_workspace_size(2 ** 31, 64) > 2 ** 38
    assert lib.lp_head_clear_status(None, None) == WORKSPACE
    assert lib.lp_head_process_workspace_size(0, 0) == 256 and lib.lp_head_process_workspace_size(4, 4000) == 256
    assert lib.lp_head_process_workspace_size(2, 2 ** 31) > 2 ** 33


def _norm(lib, x=FAKE, residual=None, w=FAKE, dtype=BF16, wdtype=BF16, T=4, H=64, xs=64, rs=64, rows=None, n=4,
          eps=1e-6, out=FAKE, odtype=BF16, os_=64, scale=None, kept=None, ks=64, ws=None, wsb=0):
    return lib.lp_head_norm(x, residual, w, dtype, wdtype, T, H, xs, rs, rows, n, eps, out, odtype, os_, scale, kept,
                            ks, ws, wsb, None)


def test_norm_refusals(lib):
    assert _norm(lib, x=None) == NULL and _norm(lib, w=None) == NULL and _norm(lib, out=None) == NULL
    assert _norm(lib, odtype=E4M3) == NULL                       # no scale
    assert _norm(lib, dtype=E4M3, wdtype=E4M3) == DTYPE and _norm(lib, dtype=99, wdtype=99) == DTYPE
    assert _norm(lib, wdtype=F16) == DTYPE and _norm(lib, odtype=F16) == DTYPE
    assert _norm(lib, T=0, n=0) == SHAPE and _norm(lib, H=0) == SHAPE and _norm(lib, n=3) == SHAPE
    assert _norm(lib, H=32769, xs=40000, os_=40000) == SHAPE
    assert _norm(lib, xs=63) == SHAPE and _norm(lib, os_=63) == SHAPE
    assert _norm(lib, residual=FAKE, rs=63) == SHAPE and _norm(lib, kept=FAKE, ks=63) == SHAPE
    assert _norm(lib, x=FAKE + 1) == SHAPE and _norm(lib, out=FAKE + 1) == SHAPE and _norm(lib, w=FAKE + 1) == SHAPE
    assert _norm(lib, eps=-1.0) == SHAPE and _norm(lib, eps=float("nan")) == SHAPE
    assert _norm(lib, rows=FAKE, n=2) == WORKSPACE               # rows are checked on the device
    assert _norm(lib, rows=FAKE, n=2, ws=FAKE, wsb=128) == WORKSPACE
    assert _norm(lib, ws=FAKE + 64, wsb=256) == WORKSPACE


def _process(lib, x=FAKE, dtype=F32, T=4, V=100, xs=100, off=None, B=4, hist=None, hoff=None, total=0, prompt=None,
             rep=None, freq=None, pres=None, bt=None, bv=None, bo=None, nb=0, mask=None, ms=4, mr=4, mi=None,
             out=FAKE * 2, os_=100, ws=FAKE, wsb=256):
    return lib.lp_head_process(x, dtype, T, V, xs, off, B, hist, hoff, total, prompt, rep, freq, pres, bt, bv, bo, nb,
                               mask, ms, mr, mi, out, os_, ws, wsb, None)


def test_process_refusals(lib):
    assert _process(lib, x=None) == NULL and _process(lib, out=None) == NULL
    assert _process(lib, hist=FAKE) == NULL and _process(lib, bt=FAKE) == NULL and _process(lib, bt=FAKE, bv=FAKE) == NULL
    assert _process(lib, ws=None) == WORKSPACE and _process(lib, wsb=255) == WORKSPACE
    assert _process(lib, ws=FAKE + 16) == WORKSPACE
    assert _process(lib, dtype=E4M3) == DTYPE
    assert _process(lib, T=0, B=0) == SHAPE and _process(lib, V=0) == SHAPE and _process(lib, B=3) == SHAPE
    assert _process(lib, xs=99) == SHAPE and _process(lib, os_=99) == SHAPE
    assert _process(lib, mask=FAKE, ms=3) == SHAPE and _process(lib, mask=FAKE, mr=3) == SHAPE
    assert _process(lib, mask=FAKE, mr=0, mi=FAKE) == SHAPE
    assert _process(lib, x=FAKE + 2) == SHAPE and _process(lib, out=FAKE + 2) == SHAPE
    assert _process(lib, out=FAKE, dtype=BF16) == SHAPE          # in place only in float32
    assert _process(lib, out=FAKE, os_=104) == SHAPE             # and with one stride


def _project(lib, x=FAKE, dtype=BF16, T=4, H=64, xs=64, sx=None, w=FAKE, V=100, wstr=64, sw=None, la=None, lb=None,
             lt=BF16, A=0, rank=0, scale=None, ids=None, off=None, B=0, out=FAKE, odtype=F32, os_=100, ws=FAKE,
             wsb=1 << 20):
    return lib.lp_head_project(x, dtype, T, H, xs, sx, w, V, wstr, sw, la, lb, lt, A, rank, scale, ids, off, B, out,
                               odtype, os_, ws, wsb, None)


def test_project_refusals(lib):
    assert _project(lib, x=None) == NULL and _project(lib, w=None) == NULL and _project(lib, out=None) == NULL
    assert _project(lib, dtype=F32) == DTYPE and _project(lib, odtype=E4M3) == DTYPE
    assert _project(lib, dtype=E4M3) == NULL and _project(lib, dtype=E4M3, sx=FAKE) == NULL     # needs both scales
    assert _project(lib, sx=FAKE) == DTYPE                       # bf16 has none
    assert _project(lib, T=0) == SHAPE and _project(lib, H=0) == SHAPE and _project(lib, V=0) == SHAPE
    assert _project(lib, H=60) == SHAPE                          # 120 bytes
    assert _project(lib, xs=68) == SHAPE and _project(lib, wstr=68) == SHAPE and _project(lib, xs=56) == SHAPE
    assert _project(lib, x=FAKE + 8) == SHAPE and _project(lib, w=FAKE + 8) == SHAPE and _project(lib, out=FAKE + 2) == SHAPE
    assert _project(lib, os_=99) == SHAPE
    a = dict(la=FAKE, lb=FAKE, A=2, rank=8, ids=FAKE, B=4)
    for missing in ("la", "lb", "ids"):
        assert _project(lib, **dict(a, **{missing: None})) == NULL
    assert _project(lib, **dict(a, rank=0)) == SHAPE and _project(lib, **dict(a, rank=65)) == SHAPE
    assert _project(lib, **dict(a, B=3)) == SHAPE and _project(lib, **dict(a, B=0)) == SHAPE
    assert _project(lib, **dict(a, lt=F16)) == DTYPE and _project(lib, **dict(a, lt=E4M3)) == DTYPE
    assert _project(lib, **dict(a, la=FAKE + 2)) == SHAPE
    assert _project(lib, ws=None) == WORKSPACE and _project(lib, ws=FAKE + 128) == WORKSPACE
    assert _project(lib, wsb=255) == WORKSPACE and _project(lib, **dict(a, wsb=256)) == WORKSPACE


def test_binding_refuses_host_tensors(lib):
    # before any pointer is read and without a GPU
    import ragged_log_probs_gb300 as lp
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.ones(8, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: lp.rms_norm(x, w), lambda: lp.rms_norm(None, w), lambda: lp.project(x, x, workspace=ws),
                 lambda: lp.process_logits(x, workspace=ws), lambda: lp.process_logits([1.0], workspace=ws),
                 lambda: lp.clear_status(ws)):
        with pytest.raises(TypeError):
            call()


def test_the_binding_is_needed(monkeypatch, tmp_path, lib):
    from ragged_log_probs_gb300 import _build, head
    monkeypatch.setattr(head, "_native", None)
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "missing.so"))
    with pytest.raises(ImportError):
        head._load()
