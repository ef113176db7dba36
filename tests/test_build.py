"""The build's order of steps (no compiler runs): the library does not need torch, and the extension is made anew for
another torch."""
import os

import pytest

from software_pipelined_tiled_pipeline_gb300 import build as gbuild


@pytest.fixture
def steps(tmp_path, monkeypatch):
    """build() with steps that only leave their files; returns what ran, in order, and a way to make the extension fail."""
    ran, fail = [], []
    for name in ("LIB", "TORCH_LIB", "TORCH_STAMP"):
        monkeypatch.setattr(gbuild, name, str(tmp_path / name))
    monkeypatch.setattr(gbuild, "BUILD", str(tmp_path))

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        what = "extension" if "TORCH_LIB" in out else "library" if "-shared" in cmd else "object"
        if what == "extension" and fail:
            r = Done()
            r.returncode, r.stderr = 1, "no headers"
            return r
        ran.append(what)
        open(out, "w").close()
        return Done()

    monkeypatch.setattr(gbuild.subprocess, "run", run)
    monkeypatch.setattr(gbuild, "check_launch_registers", lambda src, ptxas: None)
    return ran, fail


def count(ran):
    n = [ran.count(s) for s in ("object", "library", "extension")]
    ran.clear()
    return n


def test_both_are_built_once(steps):
    ran, _ = steps
    assert gbuild.build() == gbuild.LIB
    assert count(ran) == [len(gbuild.SOURCES), 1, 1]
    gbuild.build()
    assert count(ran) == [0, 0, 0]
    gbuild.build(force=True)
    assert count(ran) == [len(gbuild.SOURCES), 1, 1]


def test_the_library_needs_no_torch(steps, monkeypatch):
    ran, _ = steps
    real = gbuild.importlib.util.find_spec
    monkeypatch.setattr(gbuild.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    gbuild.build()
    assert count(ran) == [len(gbuild.SOURCES), 1, 0]
    gbuild.build()
    assert count(ran) == [0, 0, 0]
    gbuild.build(force=True)
    assert count(ran) == [len(gbuild.SOURCES), 1, 0]


def test_the_library_is_linked_where_the_extension_fails(steps):
    ran, fail = steps
    fail.append(True)
    with pytest.raises(RuntimeError, match="no headers"):
        gbuild.build()
    assert os.path.exists(gbuild.LIB) and count(ran) == [len(gbuild.SOURCES), 1, 0]
    fail.clear()
    gbuild.build()
    assert count(ran) == [0, 0, 1]


def test_another_torch_gets_another_extension(steps, monkeypatch):
    ran, _ = steps
    gbuild.build()
    count(ran)
    monkeypatch.setattr(gbuild.importlib.metadata, "version", lambda name: "0.0.1")
    gbuild.build()
    assert count(ran) == [0, 0, 1]
    gbuild.build()
    assert count(ran) == [0, 0, 0]
    os.remove(gbuild.TORCH_STAMP)
    gbuild.build()
    assert count(ran) == [0, 0, 1]
