"""What the C entries of a beam search refuse before anything runs (no GPU needed)."""
import ctypes

import pytest

import paged_mla_decode_03_gb300 as mla
from paged_mla_decode_03_gb300 import build as mla_build


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


P = 1 << 20  # an aligned address that nothing reads


def select(lib, batch=2, beams=4, k=4, vocab=100, dtype=0, end=0, logits=P, bs=400, ws=100, scores=P, finished=None,
           out=P, tokens=P, parents=P, workspace=P, nbytes=1 << 30):
    p = mla.MlaBeamParams(batch, beams, k, vocab, dtype, end)
    return lib.mla_beam_select(ctypes.byref(p), logits, bs, ws, scores, finished, out, tokens, parents, workspace, nbytes, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(beams=0), -1), (dict(k=0), -1), (dict(vocab=0), -1), (dict(dtype=3), -1), (dict(beams=65), -2),
    (dict(k=65), -2), (dict(vocab=(1 << 28) + 1), -2), (dict(batch=(1 << 20) + 1), -2), (dict(finished=P, end=-1), -1),
    (dict(finished=P, end=100), -1), (dict(logits=None), -1), (dict(scores=None), -1), (dict(out=None), -1),
    (dict(tokens=None), -1), (dict(parents=None), -1), (dict(workspace=None), -1), (dict(bs=-1), -1), (dict(ws=-1), -1),
    (dict(logits=P + 2), -4), (dict(logits=P + 1, dtype=1), -4), (dict(scores=P + 2), -4), (dict(out=P + 1), -4),
    (dict(workspace=P + 16), -4), (dict(nbytes=0), -3), (dict(batch=0, logits=None), 0)])
def test_select(lib, kw, rc):
    assert select(lib, **kw) == rc


def test_null_parameters(lib):
    assert lib.mla_beam_select(None, None, 0, 0, None, None, None, None, None, None, 0, None) == -1
    assert lib.mla_beam_workspace_size(None) == 0
    assert lib.mla_cache_reorder(None, None, 0, None, None, None, None, None, None) == -1


def reorder(lib, batch=2, beams=4, page=64, width=8, kind=0, pages=100, caches=(P,), layers=1, tables=P, lens=P, parents=P,
            spare=P, status=None):
    p = mla.MlaReorderParams(batch, beams, page, width, kind, pages)
    arr = (ctypes.c_void_p * max(1, len(caches)))(*caches) if caches is not None else None
    return lib.mla_cache_reorder(ctypes.byref(p), arr, layers, tables, lens, parents, spare, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(batch=-1), -1), (dict(beams=0), -1), (dict(width=0), -1), (dict(pages=0), -1), (dict(kind=3), -1), (dict(layers=-1), -1),
    (dict(page=16), -2), (dict(beams=65), -2), (dict(pages=1 << 31), -2), (dict(batch=1 << 23), -2), (dict(caches=None), -1),
    (dict(caches=(None,)), -1), (dict(caches=(P + 8,)), -4), (dict(tables=None), -1), (dict(lens=None), -1),
    (dict(parents=None), -1), (dict(spare=None), -1), (dict(tables=P + 2), -4), (dict(status=P + 1), -4),
    (dict(batch=0, tables=None), 0)])
def test_reorder(lib, kw, rc):
    assert reorder(lib, **kw) == rc


def test_parameter_records_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = []
    for name, cls in (("mla_beam_params", mla.MlaBeamParams), ("mla_reorder_params", mla.MlaReorderParams)):
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {f}));')
        lines.append(f'printf("%zu\\n", sizeof({name}));')
    src = tmp_path / "a.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla_decode.h"\nint main(void) {' + "".join(lines) + "}")
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "a")], check=True)
    out = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, cls in zip(out, (mla.MlaBeamParams, mla.MlaReorderParams)):
        assert [int(x) for x in line.split()] == [getattr(cls, f).offset for f, _ in cls._fields_] + [ctypes.sizeof(cls)]
