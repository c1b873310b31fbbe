"""The build: what makes the serving binding stale, and the C library on a machine
that cannot build the binding. Nothing is compiled here; the commands are
recorded."""

import os
import subprocess

import pytest

from online_softmax_attention_rf_gb300 import build


class _Done:
    returncode, stdout, stderr = 0, "", ""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the build's directories, and the list of the commands it runs."""
    for name in ("BUILD_DIR", "LIBDIR"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "LIBDIR" / "librf.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "LIBDIR" / "_rf_serving.so"))
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1'")
    (torch_dir / "include" / "ATen").mkdir(parents=True)
    monkeypatch.setattr(build, "_torch_dir", lambda: str(torch_dir))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return _Done

    monkeypatch.setattr(subprocess, "run", run)
    return tmp_path, ran


def _binding(ran):
    """The commands that made the binding."""
    return [c for c in ran if any("serving_binding" in a for a in c)]


def test_build_is_idle_when_nothing_changed(tree):
    _, ran = tree
    build.build()
    assert len(_binding(ran)) == 2 and len(ran) == len(build.sources()) + 3
    ran.clear()
    build.build()
    assert ran == []


def test_binding_is_rebuilt_for_another_torch(tree):
    tmp, ran = tree
    build.build()
    ran.clear()
    (tmp / "torch" / "version.py").write_text("__version__ = '2'")
    build.build()
    assert len(_binding(ran)) == len(ran) == 2
    ran.clear()
    build.build()
    assert ran == []


def test_binding_is_rebuilt_for_a_torch_elsewhere(tree, monkeypatch):
    tmp, ran = tree
    build.build()
    ran.clear()
    os.rename(tmp / "torch", tmp / "other")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp / "other"))
    build.build()
    assert len(_binding(ran)) == len(ran) == 2


def test_binding_is_rebuilt_for_another_python(tree, monkeypatch):
    _, ran = tree
    build.build()
    ran.clear()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "another")
    build.build()
    assert len(_binding(ran)) == len(ran) == 2


@pytest.mark.parametrize("lacking", ["torch", "torch's headers", "Python.h", "g++"])
def test_library_builds_where_the_binding_cannot(tree, monkeypatch, lacking):
    tmp, ran = tree
    if lacking == "torch":
        def none():
            raise RuntimeError("no torch")
        monkeypatch.setattr(build, "_torch_dir", none)
    elif lacking == "torch's headers":
        os.rmdir(tmp / "torch" / "include" / "ATen")
    elif lacking == "Python.h":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp / "none")})
    else:
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda n: None if n == "g++" else which(n))
    with pytest.warns(UserWarning, match="_rf_serving.so.*not built: no " + lacking.replace("+", r"\+")):
        assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert len(ran) == len(build.sources()) + 1 and not _binding(ran)


def test_library_is_linked_when_the_binding_fails(tree, monkeypatch):
    _, ran = tree
    run = subprocess.run

    def fails(cmd, **kw):
        done = run(cmd, **kw)
        if _binding([cmd]):
            done = type("Failed", (_Done,), {"returncode": 1, "stderr": "an error"})
        return done

    monkeypatch.setattr(subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="an error"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)


def test_serving_calls_raise_without_the_binding(monkeypatch, tmp_path):
    from online_softmax_attention_rf_gb300 import api
    build.build()
    monkeypatch.setattr(api, "_SERVING", None)
    monkeypatch.setattr(api._build, "BINDING_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="_rf_serving.so is not built"):
        api.draft_verify(None, None, None, None, None)
