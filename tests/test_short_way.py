"""The short way's module (binding/calls.cpp) and the library that it is bound to, on the host."""
import ctypes
import subprocess
import sys
import warnings

import pytest

import gated_deltanet_state_delta_amd._lib as L
import gated_deltanet_state_delta_amd.paged as paged
from gated_deltanet_state_delta_amd import build as B

ENTRIES = ("attn_decode", "attn_decode_workspace_size", "kv_append", "kv_read", "rope")


def _address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


def test_the_library_tells_its_header():
    assert L.load().gdn_header_digest().decode() == B.header_digest()


@pytest.mark.parametrize("digest", [b"0123456789abcdef", b"", None])
def test_a_library_of_another_header_is_refused(digest):
    """Its structs may be laid out otherwise: nothing may be called through them."""
    lib, module = L.load(), L.calls()
    text = None if digest is None else ctypes.create_string_buffer(digest)
    other = ctypes.CFUNCTYPE(ctypes.c_void_p)(lambda: text and ctypes.addressof(text))
    entries = [_address(getattr(lib, "gdn_" + name)) for name in ENTRIES]
    with pytest.raises(RuntimeError, match="different headers"):
        module.bind(_address(other), *entries)
    module.bind(_address(lib.gdn_header_digest), *entries)
    with pytest.raises(TypeError):
        module.bind(*entries)


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """A build into a folder of its own whose compilers only write their output's
    name; those whose command holds a word of the list fail."""
    fail = []

    def run(cmd, **kw):
        if any(word in arg for word in fail for arg in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "refused")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    for name in ("LIB", "CALLS", "BUILD"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    return fail


def _built(tmp_path):
    return {p.name: p.read_text() for p in tmp_path.iterdir() if p.is_file()}


@pytest.mark.parametrize("fails", ["gdn_pages.hip", "LIB.tmp"])
def test_a_build_that_fails_leaves_the_pair_as_it_was(compilers, tmp_path, fails):
    (tmp_path / "LIB").write_text("old")
    (tmp_path / "CALLS").write_text("old")
    compilers.append(fails)
    with pytest.raises(RuntimeError):
        B.build()
    assert _built(tmp_path) == {"LIB": "old", "CALLS": "old"}
    compilers.clear()
    B.build()
    assert _built(tmp_path) == {"LIB": "new", "CALLS": "new"}


@pytest.mark.parametrize("why", ["no compiler", "no headers", "no torch"])
def test_the_library_is_built_without_the_module(compilers, monkeypatch, tmp_path, capsys, why):
    """An old module beside it would be one of another header: it goes."""
    (tmp_path / "CALLS").write_text("old")
    if why == "no headers":
        compilers.append("calls.cpp")
    elif why == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        run = B.subprocess.run

        def none(cmd, **kw):
            if any("calls.cpp" in arg for arg in cmd):
                raise FileNotFoundError("g++")
            return run(cmd, **kw)
        monkeypatch.setattr(B.subprocess, "run", none)
    B.build()
    assert _built(tmp_path) == {"LIB": "new"} and "general way" in capsys.readouterr().err


@pytest.fixture
def unbound(monkeypatch):
    """As in a process that has not used the short way yet."""
    monkeypatch.setattr(L, "_calls", None)
    monkeypatch.setattr(L, "_no_calls", False)
    monkeypatch.delitem(sys.modules, L.__package__ + "._calls", raising=False)


@pytest.mark.parametrize("why", ["missing", "other torch", "other header"])
def test_without_the_module_calls_go_the_general_way(unbound, monkeypatch, tmp_path, why):
    lib = L.load()
    if why == "missing":
        monkeypatch.setattr(L, "PKG", str(tmp_path))
    elif why == "other torch":
        monkeypatch.setitem(sys.modules, L.__package__ + "._calls", None)  # importing it raises ImportError
        monkeypatch.delattr(sys.modules[L.__package__], "_calls", raising=False)
    else:
        class Other:
            gdn_header_digest = lib.gdn_version
            __getattr__ = lambda self, name: getattr(lib, name)
        monkeypatch.setattr(L, "_lib", Other())
    with pytest.warns(RuntimeWarning, match="_calls"):
        assert paged._short("rope", None) is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # one warning only
        assert paged._short("kv_append", None) is None


def test_without_the_library_there_is_no_way(unbound, monkeypatch, tmp_path):
    monkeypatch.setattr(L, "_lib", None)
    monkeypatch.setattr(L, "LIB_PATH", str(tmp_path / "libgdn.so"))
    with pytest.raises(Exception):
        paged._short("rope", None)
    assert not L._no_calls
