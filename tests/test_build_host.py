"""When the library and the binding's extension are built again, and when the extension is not loaded."""
import os

import pytest
import torch

import __graft_entry__
from w6a8_quantized_linear_gb300 import build, qlin


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build of its own: files as old as their names' order says, the newest built."""
    for i, (name, file) in enumerate((("BINDING_SOURCE", "binding.cpp"), ("HEADER", "qlin.h"), ("LIB", "lib.so"), ("BINDING", "binding.so"),
                                      ("STAMP", "binding.so.torch"))):
        path = tmp_path / file
        path.write_text(build.stamp() if name == "STAMP" else "")
        os.utime(path, (1000 + i, 1000 + i))
        monkeypatch.setattr(build, name, str(path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", [build.HEADER])
    monkeypatch.setattr(build, "UNITS", [])
    return monkeypatch


def test_the_extension_is_older_than_what_it_is_made_of(tree):
    assert build.up_to_date()
    for newer in ("BINDING_SOURCE", "HEADER"):
        before = os.path.getmtime(getattr(build, newer))
        os.utime(build.LIB, (3000, 3000))
        os.utime(getattr(build, newer), (2000, 2000))
        assert not build.up_to_date(), newer
        os.utime(getattr(build, newer), (before, before))
    assert build.up_to_date()
    os.utime(build.HEADER, (4000, 4000))
    assert not build.up_to_date()


@pytest.mark.parametrize("change", ["torch", "no stamp", "no extension"])
def test_an_extension_of_another_torch_is_built_again(tree, change):
    assert build.up_to_date() and build.binding_fits()
    if change == "torch":
        tree.setattr(torch, "__version__", "1.0")
    else:
        os.remove(build.STAMP if change == "no stamp" else build.BINDING)
    assert not build.up_to_date()
    assert change == "no extension" or not build.binding_fits()


def test_a_build_that_ends_between_the_library_and_the_extension_is_not_taken_for_whole(tree):
    class Done:
        returncode, stdout, stderr = 0, "", ""

        def __init__(self, cmd, **kw):
            self.cmd = cmd

        def communicate(self):
            return "", ""

    def link(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done(cmd)

    def fails(obj, tag):
        raise RuntimeError("linking the binding failed")

    tree.setattr(build.subprocess, "Popen", Done)
    tree.setattr(build.subprocess, "run", link)
    tree.setattr(build, "_link_binding", fails)
    with pytest.raises(RuntimeError, match="linking"):
        build.build_library(force=True)
    assert os.path.getmtime(build.LIB) > 10000  # replaced
    assert not build.up_to_date() and not build.binding_fits()


def test_what_takes_an_extensions_place_refers_every_call_to_the_other_way(tmp_path, monkeypatch):
    __graft_entry__.build()
    monkeypatch.setattr(qlin, "_binding", None)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_qlin_binding.so"))
    with pytest.warns(RuntimeWarning, match="_qlin_binding"):
        binding = qlin._load_binding()
    assert qlin._load_binding() is binding
    for call in ("kv_append", "kv_weigh", "kv_evict", "adjust_logits"):
        assert getattr(binding, call)(0, 1, None) is None


def test_two_builds_at_once_do_not_trip_over_the_stamp(tree):
    class Done:
        returncode, stdout, stderr = 0, "", ""

        def __init__(self, cmd, **kw):
            pass

        def communicate(self):
            return "", ""

    def link(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done(cmd)

    exists = os.path.exists  # the other build takes the stamp away between a look and a step
    tree.setattr(os.path, "exists", lambda p: True if p == build.STAMP else exists(p))
    os.remove(build.STAMP)
    tree.setattr(build.subprocess, "Popen", Done)
    tree.setattr(build.subprocess, "run", link)
    tree.setattr(build, "_link_binding", lambda obj, tag: "")
    build.build_library(force=True)
    assert build.binding_fits()
