"""What the build step makes and when, with a compiler that only writes its output's
name: no torch, a failing host compile, torch versions in turn."""
import importlib.metadata
import importlib.util
import os
import subprocess
import time

import pytest

from int4_grouped_gemm_gb300 import build


@pytest.fixture
def steps(tmp_path, monkeypatch):
    """The commands of each build into tmp_path; every output comes a second after the last."""
    commands, clock = [], [time.time() + 1000]

    def fake(cmd, **_):
        commands.append(cmd)
        if getattr(fake, "fails", None) and any(fake.fails in c for c in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "refused")
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        clock[0] += 1
        os.utime(out, (clock[0], clock[0]))
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_native.so"))
    monkeypatch.setattr(subprocess, "run", fake)

    def run(**kw):
        commands.clear()
        build.build(**kw)
        return [c[c.index("-o") + 1] for c in commands]
    run.fake, run.commands = fake, commands
    return run


def test_the_library_needs_no_torch(steps, monkeypatch):
    find, version = importlib.util.find_spec, importlib.metadata.version

    def none(name, *a):
        return None if name == "torch" else find(name, *a)

    def absent(name):
        if name == "torch":
            raise importlib.metadata.PackageNotFoundError(name)
        return version(name)
    monkeypatch.setattr(importlib.util, "find_spec", none)
    monkeypatch.setattr(importlib.metadata, "version", absent)
    made = steps()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert sum(o.endswith(".o") for o in made) == len(build.SOURCES)
    assert steps() == []


def test_no_compiler_but_nvcc_is_called(steps):
    steps()
    assert os.path.exists(build.BINDING)
    assert {c[0] for c in steps.commands} == {build.nvcc()}


def test_the_library_is_made_even_if_the_module_is_not(steps):
    steps.fake.fails = "binding.cpp"
    with pytest.raises(RuntimeError, match="refused"):
        steps()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_the_module_follows_the_torch_version(steps, monkeypatch):
    """Back at a version whose object is there already, older than the module of the
    version between: linked again, and nothing is compiled."""
    current = ["2.9.1"]
    monkeypatch.setattr(importlib.metadata, "version", lambda name: current[0])

    def linked():
        with open(build.BINDING) as f:
            return f.read()
    steps()
    first = linked()
    assert "2.9.1" in first
    current[0] = "2.11.0"
    made = steps()
    assert len(made) == 2 and "2.11.0" in linked()          # its object and the module
    current[0] = "2.9.1"
    made = steps()
    assert len(made) == 1 and "2.9.1" in linked() and "2.11.0" not in linked()
    assert steps() == []


def test_the_module_follows_the_python_version(steps, monkeypatch):
    steps()
    get = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda n: ".cpython-399-none.so" if n == "EXT_SUFFIX" else get(n))
    assert len(steps()) == 2
    assert steps() == []
