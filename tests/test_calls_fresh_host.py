"""A compiled module of csrc/binding.cpp belongs to one torch, one Python and one
include/qgemv.h: with others it is another file, or out of date.  No GPU."""
import importlib.metadata
import os
import sysconfig

import pytest

from block_quantized_gemv_quantize_gb300 import build


def test_another_torch_or_python_is_another_file(monkeypatch):
    here = build.calls_path()
    assert os.path.dirname(here) == build.BUILD and here == build.calls_path() == build.CALLS
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "9.9.9+cu999")
        other_torch = build.calls_path()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: {"SOABI": "cpython-399-other"}.get(name))
        other_python = build.calls_path()
    assert len({here, other_torch, other_python}) == 3


@pytest.mark.parametrize("name", ["binding.cpp", "qgemv.h", "build.py"])
def test_a_module_older_than_what_it_is_made_of_is_out_of_date(monkeypatch, tmp_path, name):
    assert name in [os.path.basename(f) for f in build.calls_deps()]
    path, newer = tmp_path / "calls.so", tmp_path / name
    path.write_bytes(b"")
    newer.write_bytes(b"")
    monkeypatch.setattr(build, "calls_deps", lambda: [str(newer)])
    os.utime(path, (2000, 2000))
    os.utime(newer, (1000, 1000))
    assert build.calls_up_to_date(str(path))
    os.utime(newer, (3000, 3000))
    assert not build.calls_up_to_date(str(path))
    assert not build.calls_up_to_date(str(tmp_path / "absent.so"))


def test_the_entry_points_types_come_from_the_header():
    src = open(os.path.join(build.CSRC, "binding.cpp")).read()
    for name in ("kv_write", "kv_read", "attn_paged", "kv_page_bytes", "attn_paged_workspace_bytes"):
        assert f"decltype(&::{name})" in src
