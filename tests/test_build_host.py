"""The checked library's build (no compiler needed: commands are recorded and their outputs touched): what
it links is compiled anew when that is asked for, and flags of its own stay out of the ordinary objects."""
import os

import pytest

from fft_signal_processing_gb300 import _build


@pytest.fixture
def compiled(tmp_path, monkeypatch):
    """Objects in a folder of their own; returns a function that builds and tells what was compiled."""
    for name in ("OBJ", "OBJ_CHECKED", "LIB", "LIB_CHECKED"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    done = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        if "-c" in cmd:
            done.append(cmd)

        class Result:
            returncode, stdout, stderr = 0, "", ""
        return Result()

    monkeypatch.setattr(_build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(_build.subprocess, "run", run)

    def build(**k):
        done.clear()
        _build.build(**k)
        return {os.path.basename(c[c.index("-c") + 1]) for c in done}
    return build


def test_checked_library_shares_objects_without_checks(compiled):
    everything = compiled()
    assert "gnorm.cu" in everything and "shift.cu" in everything
    assert compiled() == set()
    checked = compiled(checked=True)
    assert "shift.cu" in checked and "gnorm.cu" not in checked and "linattn_api.cu" not in checked
    assert compiled(checked=True) == set()


def test_force_compiles_all_that_is_linked(compiled):
    everything = compiled()
    compiled(checked=True)
    assert compiled(checked=True, force=True) == everything
    assert compiled(force=True) == everything


def test_flags_stay_out_of_the_ordinary_objects(compiled):
    everything = compiled()
    assert compiled(checked=True, extra=["-DMORE"]) == everything
    for name in os.listdir(_build.OBJ):
        assert "-DMORE" not in open(os.path.join(_build.OBJ, name)).read(), name
    assert compiled() == set()
