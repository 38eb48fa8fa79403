"""When the library and its Python binding are rebuilt: after a change of torch or of Python, of flags, of sources.  Compilers are
stood in for by a function that writes the output file."""
import os
import types

import pytest
import torch

from kv_cache_vector_norm_b200 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of empty sources in a folder of its own, and the list of the commands that were run."""
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir(), include.mkdir()
    names = {n for src, (_, deps) in _build.UNITS.items() for n in (src, *deps)} | {"tq_internal.h", _build.BIND_SOURCE}
    for f in [csrc / n for n in names] + [include / "tq.h"]:
        f.write_text("")
        os.utime(f, (1000, 1000))
    for name, at in dict(PKG=tmp_path, CSRC=csrc, INCLUDE=include, LIB=tmp_path / "libtq.so", BIND=tmp_path / "_bind.so",
                         BIND_STAMP=tmp_path / "_bind.stamp", BUILD_DIR=tmp_path / "_build",
                         LIB_FLAGS=tmp_path / "_build" / "libtq.flags").items():
        monkeypatch.setattr(_build, name, str(at))
    ran = []

    def compiler(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("")
        return types.SimpleNamespace(returncode=0, stdout="", communicate=lambda: ("", None))

    monkeypatch.setattr(_build.subprocess, "Popen", compiler)
    monkeypatch.setattr(_build.subprocess, "run", compiler)
    tree = types.SimpleNamespace(path=tmp_path, ran=ran)
    tree.sources = lambda: [os.path.basename(a) for c in ran for a in c if a.endswith((".cu", ".cpp"))]
    return tree


def test_nothing_is_built_twice(tree):
    assert _build.needs_build()
    _build.build()
    assert sorted(tree.sources()) == sorted([*_build.UNITS, _build.BIND_SOURCE]) and not _build.needs_build()
    tree.ran.clear()
    _build.build()
    assert not tree.ran


@pytest.mark.parametrize("what", ["torch", "python", "stamp"])
def test_another_torch_or_python_rebuilds_the_binding_alone(tree, monkeypatch, what):
    _build.build()
    tree.ran.clear()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif what == "python":
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-00")
    else:
        os.remove(_build.BIND_STAMP)
    assert _build.needs_build()
    _build.build()
    assert tree.sources() == [_build.BIND_SOURCE] and not _build.needs_build()


def test_objects_of_other_flags_are_not_linked_in(tree):
    _build.build()
    tree.ran.clear()
    _build.build(extra=("-DSOMETHING",))
    cu = [n for n, (kind, _) in _build.UNITS.items() if kind == "cu"]
    assert sorted(tree.sources()) == sorted(cu) and all("-DSOMETHING" in c for c in tree.ran if "-c" in c)
    assert _build.needs_build()
    tree.ran.clear()
    _build.build()
    assert sorted(tree.sources()) == sorted(cu) and not any("-DSOMETHING" in c for c in tree.ran) and not _build.needs_build()


def test_a_source_rebuilds_what_is_made_of_it(tree):
    _build.build()
    for name, want in (("tq_pages_kernels.cuh", ["tq_pages.cu"]), ("tq_bind.cpp", ["tq_bind.cpp"]),
                       ("tq_internal.h", sorted(_build.UNITS))):
        tree.ran.clear()
        soon = 10 + max(os.path.getmtime(os.path.join(d, f)) for d, _, fs in os.walk(tree.path) for f in fs)
        os.utime(tree.path / "csrc" / name, (soon, soon))
        assert _build.needs_build()
        _build.build()
        assert sorted(tree.sources()) == want
        for d, _, fs in os.walk(tree.path):             # as if all of it had been built after the change
            for f in fs:
                if d != str(tree.path / "csrc"):
                    os.utime(os.path.join(d, f), (soon + 1, soon + 1))


def test_a_library_without_its_objects_is_taken_as_it_is(tree):
    """The built files alone, as they are carried to another machine: no compiler runs."""
    _build.build()
    for f in os.listdir(_build.BUILD_DIR):
        os.remove(os.path.join(_build.BUILD_DIR, f))
    assert not _build.needs_build()
