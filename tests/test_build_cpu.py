"""What the build makes where torch or its headers are not there: the compiler's commands are
only written down, and what they would have written is there afterwards."""
import os

import pytest

from int4_weight_only_moe_gb300 import _build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    ran = []

    def run(cmd):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            return ""

    monkeypatch.setattr(_build, "_run", run)
    for name, path in (("BUILD", "build"), ("LIBDIR", "lib"), ("LIB", "lib/libmoe_w4a16.so"), ("CALLS", "lib/moe_w4a16_calls.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / path))
    return ran


def compilers(ran):
    return [os.path.basename(c[0]) for c in ran]


def test_the_library_needs_nvcc_alone(commands, monkeypatch):
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    assert not _build.up_to_date()
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB) and not os.path.exists(_build.CALLS)
    assert set(compilers(commands)) == {"nvcc"} and len(commands) == len(_build.SOURCES) + 1
    assert _build.up_to_date()
    commands.clear()
    assert _build.build() == _build.LIB and not commands


@pytest.mark.parametrize("step", ["-c", "-shared"])
def test_an_extension_that_cannot_be_built_leaves_the_library(commands, monkeypatch, step):
    run = _build._run

    def fails(cmd):
        if cmd[0] == "g++" and step in cmd:
            raise RuntimeError("command failed: no Python.h")
        return run(cmd)

    monkeypatch.setattr(_build, "_run", fails)
    os.makedirs(_build.LIBDIR)
    with open(_build.CALLS, "w"):
        os.utime(_build.CALLS, (0, 0))  # (of an older source)
    with pytest.warns(UserWarning, match="no Python.h"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.CALLS) and not _build.up_to_date()
    # it is tried again, and alone
    commands.clear()
    monkeypatch.setattr(_build, "_run", run)
    _build.build()
    assert compilers(commands) == ["g++", "g++"] and _build.up_to_date()


def test_each_is_built_for_its_own_sources(commands):
    _build.build()
    assert compilers(commands).count("g++") == 2
    now = os.path.getmtime(_build.LIB)
    for target, want in ((_build.CALLS, {"g++"}), (_build.LIB, {"nvcc"})):
        commands.clear()
        os.utime(target, (now - 1e9, now - 1e9))
        assert not _build.up_to_date()
        _build.build()
        assert set(compilers(commands)) == want and _build.up_to_date()
