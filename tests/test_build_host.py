"""What build.py makes, and when it makes it again, with the compilers replaced by a stand-in."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py with its outputs under tmp_path; build.runs counts the commands, each of which writes its -o file."""
    spec = importlib.util.spec_from_file_location("skv_build_under_test", os.path.join(ROOT, "split_kv_merge_b200", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.BUILD, m.LIB, m.BINDING = str(tmp_path / "o"), str(tmp_path / "lib.so"), str(tmp_path / "_serving.so")
    m.runs = []

    def run(cmd, **kw):
        m.runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(m.subprocess, "run", run)
    m.bindings = lambda: sum(m.BINDING in c for c in m.runs)
    return m


def test_the_library_needs_no_torch(build, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert build.bindings() == 0 and "not built" in capsys.readouterr().err


def test_the_extension_is_made_again_for_another_torch(build, tmp_path, monkeypatch):
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    spec = importlib.util.spec_from_file_location("torch", torch / "__init__.py")
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: spec)
    for want in (1, 1):
        build.build()
        assert build.bindings() == want
    (torch / "version.py").write_text("__version__ = '2'\n")
    os.utime(torch / "version.py", (1, 1))         # an older release installed over it
    for want in (2, 2):
        build.build()
        assert build.bindings() == want
