"""When the decode-step binding is compiled and linked again (the commands are a stand-in's)."""

import os

import pytest
import torch

from fp8_grouped_expert_gb300 import build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The commands run, in a build tree of its own; each makes its output, a second later than
    the one before."""
    ran, clock = [], [os.path.getmtime(build.__file__) + 1e6]

    def run(cmd):
        target = cmd[cmd.index("-o") + 1]
        with open(target, "w") as f:
            f.write(" ".join(cmd))
        clock[0] += 1
        os.utime(target, (clock[0], clock[0]))
        ran.append("link" if "-shared" in cmd else "compile")
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_decode.so"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfge.so"))
    run(["-shared", "-o", build.LIB])
    ran.clear()
    return ran


def _build():
    build.link_binding(build.compile_binding())
    with open(build.BINDING) as f:
        return f.read()


def test_nothing_is_done_twice(commands):
    _build()
    assert commands == ["compile", "link"]
    _build()
    assert commands == ["compile", "link"]


def test_another_torch_links_its_own(commands, monkeypatch):
    linked = {}
    for version in ("2.1", "2.2"):
        monkeypatch.setattr(torch, "__version__", version)
        linked[version] = _build()
    assert commands == ["compile", "link"] * 2 and linked["2.1"] != linked["2.2"]
    # back again: the object is there, but what is linked is the other's
    commands.clear()
    monkeypatch.setattr(torch, "__version__", "2.1")
    assert _build() == linked["2.1"] and commands == ["link"]
    assert _build() == linked["2.1"] and commands == ["link"]
