"""The compiled short way into the paged cache's calls (csrc/binding.cpp) is an
addition: the library builds, and the package imports and calls it, where that
module cannot be compiled or loaded.  No GPU."""
import pytest

from block_quantized_gemv_quantize_gb300 import build

TINY = 'extern "C" int answer() { return 42; }\n'


@pytest.fixture
def no_headers(monkeypatch):
    def fail(force=False):
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(build, "build_calls", fail)


def test_the_library_builds_without_the_module(no_headers, monkeypatch, tmp_path, capsys):
    src = tmp_path / "tiny.cu"
    src.write_text(TINY)
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "out" / "libtiny.so"))
    import ctypes

    assert ctypes.CDLL(build.build(force=True)).answer() == 42
    assert "No module named 'torch'" in capsys.readouterr().err


def test_an_up_to_date_library_needs_no_module(no_headers, monkeypatch):
    monkeypatch.setattr(build, "up_to_date", lambda lib=None: True)
    assert build.build() == build.LIB


@pytest.mark.parametrize("content", [None, b"no library"])
def test_without_the_module_the_calls_go_through_ctypes(monkeypatch, tmp_path, content):
    from block_quantized_gemv_quantize_gb300 import _lib

    path = tmp_path / "calls.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(build, "CALLS", str(path))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        calls = _lib._load_calls()
    assert calls.kv_write() is calls.kv_read() is calls.attn_paged() is None
