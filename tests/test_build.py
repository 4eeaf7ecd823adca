"""CPU tests of the build's order: the HIP library needs neither torch's headers nor a host compiler."""
import os

import pytest

from fp8_moe_grouped_amd import build as B


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The commands that a build runs, without running them; results go to a folder of the test."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "calls.so"))
    return ran


def test_every_source_is_compiled_and_linked(commands):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.CALLS)
    assert sum("-c" in c for c in commands) == len(B.SOURCES)


@pytest.mark.parametrize("error", [RuntimeError("command failed (127): g++"), ImportError("no module torch"),
                                   FileNotFoundError("g++")])
def test_library_without_the_extension(commands, monkeypatch, error):
    """The extension's failure is reported, after the library is linked."""
    def fail():
        raise error

    monkeypatch.setattr(B, "build_calls", fail)
    with pytest.raises(type(error)) as e:
        B.build()
    assert e.value is error and os.path.exists(B.LIB) and not os.path.exists(B.CALLS)


def test_failed_source_is_reported(commands, monkeypatch):
    run = B._run

    def broken(cmd):
        if any(str(a).endswith("route.hip") for a in cmd):
            raise RuntimeError("command failed (1): route.hip")
        return run(cmd)

    monkeypatch.setattr(B, "_run", broken)
    with pytest.raises(RuntimeError, match="route.hip"):
        B.build()
    assert not os.path.exists(B.LIB)
