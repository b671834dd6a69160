"""The library without the extension module that marshals calls (no GPU needed)."""
import ctypes
import os
import warnings

import pytest
import torch

import tiled_online_softmax_02_gb300 as attn
from tiled_online_softmax_02_gb300 import _binding, build


@pytest.fixture
def unloaded(monkeypatch):
    """The binding as it is before its first call, to be left as it was."""
    build.build()
    monkeypatch.setattr(_binding, "_lib", None)
    monkeypatch.setattr(_binding, "_calls", None)


def test_a_library_without_the_module(unloaded, monkeypatch, tmp_path):
    """Loads, says so once, and every call is marshalled in Python."""
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning, match="none.so"):
        lib = attn.load_library()
    assert lib.attn_version() == 100
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert attn.load_library() is lib
    # the checks of the Python side answer: these are CPU tensors
    c, s = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2, 16, 4), dtype=torch.uint8)
    x, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int64)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    for call in (lambda: attn.attn_cache_append_fp4(x, x, slots, c, c.clone(), s, s.clone()),
                 lambda: attn.attn_cache_read_fp4(c, c, s, s, slots),
                 lambda: attn.attn_fwd_paged_fp4(x.half(), c, c, s, s, i32(1, 2), i32(2), i32(1)),
                 lambda: attn.attn_rope(x, x, torch.ones(32, dtype=torch.float64), positions=i32(3))):
        with pytest.raises(ValueError):
            call()


def test_a_module_that_cannot_be_loaded(unloaded, monkeypatch, tmp_path):
    bad = tmp_path / "bad.so"
    bad.write_bytes(b"no library")
    monkeypatch.setattr(build, "CALLS", str(bad))
    with pytest.warns(RuntimeWarning, match="bad.so"):
        assert attn.load_library().attn_version() == 100


def test_the_module_is_taken_where_it_is(unloaded):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        attn.load_library()
    assert _binding._calls is not _binding._NoCalls and _binding._calls.append() is None


def test_a_module_that_cannot_be_compiled(monkeypatch, tmp_path):
    """The build warns with the compiler's words, leaves no module of other sources, and the library stays."""
    build.build()
    calls = tmp_path / "calls.so"
    calls.write_bytes(b"of older sources")
    os.utime(calls, (0, 0))
    src = tmp_path / "src"
    src.mkdir()
    (src / "calls.cpp").write_text("#error cannot be compiled here\n")
    monkeypatch.setattr(build, "CALLS", str(calls))
    monkeypatch.setattr(build, "_library_up_to_date", lambda: True)
    monkeypatch.setattr(build, "CSRC", str(src))
    before = os.path.getmtime(build.LIB)
    with pytest.warns(RuntimeWarning, match="cannot be compiled here"):
        assert build.build() == build.LIB
    assert not calls.exists() and os.path.getmtime(build.LIB) == before
    assert ctypes.CDLL(build.LIB).attn_version() == 100


def test_a_build_without_a_compiler(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build, "_library_up_to_date", lambda: True)
    monkeypatch.setenv("PATH", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="was not built"):
        build.build()
