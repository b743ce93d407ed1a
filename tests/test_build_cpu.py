"""What the build makes where torch or its headers are not there: the compiler's commands are
only written down, and what they would have written is there afterwards."""
import os
import time
from concurrent.futures import ThreadPoolExecutor

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


def test_another_torch_or_python_builds_the_extension_again(commands, monkeypatch):
    import torch
    assert _build._version(os.path.dirname(torch.__file__)) == torch.__version__
    _build.build()
    with open(_build.CALLS + ".txt") as f:
        assert torch.__version__ in f.read()
    for name, what in (("_version", lambda path: "1.2.3"), ("built_for", lambda version: f"{version}, another Python")):
        commands.clear()
        monkeypatch.setattr(_build, name, what)
        assert not _build.up_to_date()
        _build.build()
        assert compilers(commands) == ["g++", "g++"] and _build.up_to_date()


def test_builds_at_once_wait_for_one_another(commands, monkeypatch):
    run, here = _build._run, []

    def slowly(cmd):
        linking = cmd[0] != "g++" and "-shared" in cmd
        if linking:
            here.append(1)
            time.sleep(0.2)
            assert len(here) == 1, "two builds link into one file"
        out = run(cmd)
        if linking:
            here.pop()
        return out

    monkeypatch.setattr(_build, "_run", slowly)
    with ThreadPoolExecutor(4) as pool:
        for made in [pool.submit(_build.build) for _ in range(4)]:
            assert made.result() == _build.LIB
    assert len(commands) == len(_build.SOURCES) + 3  # (one of them built)


def test_what_is_up_to_date_writes_nothing(commands, monkeypatch, tmp_path):
    _build.build()
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "nowhere"))
    assert _build.build() == _build.LIB and not os.path.exists(_build.BUILD)


# ---------------------------------------------------------------- loading what was built


@pytest.fixture
def extension(monkeypatch, tmp_path):
    """A file in the extension's place, of a text that is no library."""
    from int4_weight_only_moe_gb300 import _calls
    monkeypatch.setattr(_calls, "module", None)
    monkeypatch.setattr(_calls, "_refused", None, raising=False)
    monkeypatch.setattr(_calls, "PATH", str(tmp_path / "moe_w4a16_calls.so"))
    with open(_calls.PATH, "w") as f:
        f.write("no library")
    return _calls


def gather_by_steps(monkeypatch):
    """A call with a given output, which asks for the extension, on tensors that only say where
    they are: whether it has gone to the C entry of the Python steps."""
    from int4_weight_only_moe_gb300 import dispatch
    from tests import test_dispatch_devices_cpu as t
    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0

    monkeypatch.setattr(dispatch, "lib", Lib)
    monkeypatch.setattr(dispatch, "_order_rows", lambda m, k, e, b: m * k + min(e, m * k) * (b - 1))
    monkeypatch.setattr(t.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(t.torch._C, "_cuda_getCurrentRawStream", lambda dev: 7, raising=False)
    t.CALLS["gather"][0](t.new("gather"))
    return launched == ["moe_w4a16_dispatch_gather"]


@pytest.mark.parametrize("note", [None, "torch 1.2.3, Python .so\n", "right"])
def test_an_extension_that_does_not_load_leaves_the_python_steps(extension, monkeypatch, note):
    import torch
    if note:
        with open(extension.PATH + ".txt", "w") as f:
            f.write(extension.built_for(torch.__version__) if note == "right" else note)
    with pytest.warns(UserWarning, match="Python steps"):
        assert extension.load() is None
    import warnings
    with warnings.catch_warnings():  # (said once)
        warnings.simplefilter("error")
        assert extension.load() is None and extension.module is None
        assert gather_by_steps(monkeypatch)
    os.utime(extension.PATH, ns=(1, 1))  # another file there is tried
    with pytest.warns(UserWarning, match="Python steps"):
        assert extension.load() is None


def test_what_was_built_here_is_loaded(monkeypatch):
    import __graft_entry__
    from int4_weight_only_moe_gb300 import _calls
    __graft_entry__.build()
    monkeypatch.setattr(_calls, "module", None)
    assert _calls.load() is not None and _calls.load() is _calls.module
