"""The build: the library needs no torch and no host compiler for the quick argument checks, which follow the installed torch."""

import os
import stat
import types
import warnings

import pytest

from memory_bound_gemv_gb300 import build, decode

torch = pytest.importorskip("torch")


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one tiny source, in a folder of its own."""
    source = tmp_path / "one.cu"
    source.write_text('extern "C" int one() { return 1; }\n')
    made = tmp_path / "made"
    for name, value in (("BUILD", made), ("LIB", made / "lib.so"), ("BINDING", made / "binding.so")):
        monkeypatch.setattr(build, name, str(value))
    monkeypatch.setattr(build, "_sources", lambda: [str(source)])
    return made


def compiler(tmp_path, monkeypatch, text):
    path = tmp_path / "compiler"
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("CXX", str(path))


WRITES = 'while [ "$1" != "-o" ]; do shift; done\necho made >> "$2"\n'


@pytest.mark.parametrize("text", ["exit 1\n", WRITES + "exit 1\n", None])
def test_the_library_is_built_where_the_quick_form_cannot_be(small, tmp_path, monkeypatch, capsys, text):
    if text is None:
        monkeypatch.setenv("CXX", str(tmp_path / "no such compiler"))
    else:
        compiler(tmp_path, monkeypatch, text)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert build.up_to_date() and not build.binding_up_to_date()
    assert "checks" in capsys.readouterr().err
    assert not [f for f in os.listdir(small) if f.endswith(".tmp")]
    when = os.path.getmtime(build.LIB)
    build.build()
    assert os.path.getmtime(build.LIB) == when  # only what is missing is tried again


def test_another_torch_makes_the_quick_form_stale(small, tmp_path, monkeypatch):
    compiler(tmp_path, monkeypatch, WRITES)
    build.build()
    assert build.up_to_date() and build.binding_up_to_date()
    when = os.path.getmtime(build.LIB)
    with open(build.BINDING + ".torch", "w") as f:
        f.write("1.0")
    assert not build.binding_up_to_date()
    build.build()
    assert build.binding_up_to_date() and os.path.getmtime(build.LIB) == when
    os.remove(build.BINDING)
    assert not build.binding_up_to_date()


def test_the_torch_version_is_read_without_an_import():
    assert build._torch_version() == torch.__version__


def test_calls_go_the_python_way_without_the_quick_form(tmp_path, monkeypatch):
    with pytest.warns(UserWarning, match="in Python"):  # made for another torch
        quick = decode._load_binding(types.SimpleNamespace(__version__="1.0"))
    assert quick.attn(1, 2) == quick.norm() == -1
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "missing.so"))

    def fails(*args, **kw):
        raise RuntimeError("no compiler")

    monkeypatch.setattr(build, "build", fails)
    with pytest.warns(UserWarning, match="no compiler"):
        assert decode._load_binding(torch).rope() == -1


def test_the_quick_form_is_the_one_in_use():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert decode._load_binding(torch).torch_version == torch.__version__
