"""What the build compiles and links again, with a compiler that only writes its
outputs."""
import os
import subprocess
import sys
import types

import pytest
import torch

from diffusion_draft_tree_gb300 import _build


@pytest.fixture
def builds(tmp_path, monkeypatch):
    """Runs the build in an empty place; returns the commands of each run."""
    ran = []

    def fake(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        ran.append(cmd)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libddtree.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_ddtree.so"))
    monkeypatch.setattr(subprocess, "run", fake)

    def build(version):
        monkeypatch.setattr(torch, "__version__", version)
        ran.clear()
        _build.build()
        return list(ran)

    return build


def _linked_from():
    with open(_build.BINDING) as f:
        return next(os.path.basename(x) for x in f.read().split() if "binding." in x)


def test_nothing_is_built_twice(builds):
    assert len(builds("2.0")) == len(_build.SOURCES) + 3  # objects, the module's, two links
    assert builds("2.0") == []


def test_the_module_follows_the_torch_it_is_loaded_with(builds):
    builds("2.0")
    first = _linked_from()
    assert len(builds("3.0")) == 2 and _linked_from() != first
    assert len(builds("2.0")) == 1 and _linked_from() == first  # (its object is still there)
    assert builds("2.0") == []


def test_the_module_follows_the_interpreter(builds, monkeypatch):
    builds("2.0")
    first = _linked_from()
    real = _build.sysconfig.get_config_var
    monkeypatch.setattr(_build.sysconfig, "get_config_var",
                        lambda name: "other-abi" if name == "SOABI" else real(name))
    assert len(builds("2.0")) == 2 and _linked_from() != first


def test_a_link_that_fails_is_done_again(builds, monkeypatch):
    builds("2.0")
    good = subprocess.run

    def broken(cmd, **kw):
        r = good(cmd, **kw)
        r.returncode = int("-shared" in cmd)
        return r

    monkeypatch.setattr(subprocess, "run", broken)
    with pytest.raises(RuntimeError, match="link of _ddtree.so"):
        builds("3.0")
    monkeypatch.setattr(subprocess, "run", good)
    assert len(builds("2.0")) == 1


def test_a_module_of_another_torch_is_refused():
    code = ("import torch; torch.__version__ = '1.0'\n"
            "import diffusion_draft_tree_gb300.ops")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode and "built for another torch" in r.stderr
