"""What the build compiles again, with a compiler that only records its calls."""
import os

import pytest

from long_context_recsa_b200 import build as B


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """build() in a folder of its own; returns the sources and outputs of each compiler call."""
    made = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        if "-c" in cmd:
            with open(cmd[cmd.index("-MF") + 1], "w") as f:
                f.write("x.o: " + cmd[-1])
            made.append(os.path.basename(cmd[-1]))
        else:
            made.append("link")

    monkeypatch.setattr(B, "OUT", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "OUT_BOUNDS", str(tmp_path / "lib_bounds.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(B.subprocess, "run", run)

    def build(**kw):
        made.clear()
        B.build(**kw)
        return sorted(made)

    return build


def test_nothing_is_made_twice(calls):
    every = sorted([*B.SOURCES, "link"])
    assert calls() == every
    assert calls() == []
    assert calls(force=True) == every
    assert calls(debug_bounds=True) == every             # objects of its own
    assert calls() == [] and calls(debug_bounds=True) == []


def test_other_flags_or_sources_make_the_objects_anew(calls, monkeypatch):
    every = sorted([*B.SOURCES, "link"])
    calls()
    monkeypatch.setattr(B, "ARCH", [*B.ARCH, "-DOTHER"])
    assert calls() == every
    assert calls() == []
    monkeypatch.setattr(B, "SOURCES", B.SOURCES[:-1])
    assert calls() == sorted([*B.SOURCES, "link"])


def test_a_build_that_failed_is_taken_up_again(calls, monkeypatch):
    calls()
    monkeypatch.setattr(B, "ARCH", [*B.ARCH, "-DOTHER"])
    run = B.subprocess.run

    def fail(cmd, check):
        if cmd[-1].endswith(B.SOURCES[-1]):
            raise OSError("no compiler")
        run(cmd, check)

    monkeypatch.setattr(B.subprocess, "run", fail)
    with pytest.raises(OSError):
        calls()
    monkeypatch.setattr(B.subprocess, "run", run)
    assert B.SOURCES[-1] in calls()
