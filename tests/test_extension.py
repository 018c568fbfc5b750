"""The Python extension beside libkda.so: its file names the interpreter it is built for, and
a build that cannot make it leaves what was built before."""
import os
import subprocess
import sysconfig
import types

import pytest

from gated_delta_rule_35_amd import binding, build


def test_the_file_names_its_interpreter():
    binding._load_caller()
    from gated_delta_rule_35_amd import _kda_py
    assert _kda_py.__file__ == build.CALLER
    assert os.path.basename(build.CALLER) == "_kda_py" + sysconfig.get_config_var("EXT_SUFFIX")
    assert "cpython" in build.CALLER


@pytest.mark.parametrize("fails", ["gcc", "hipcc"])
def test_a_failed_build_leaves_the_last_one(fails, monkeypatch, tmp_path):
    for name in ("LIB", "CALLER"):
        path = tmp_path / name
        path.write_text("old")
        monkeypatch.setattr(build, name, str(path))

    def run(cmd, **kw):
        if fails in os.path.basename(cmd[0]):
            if kw.get("check"):
                raise subprocess.CalledProcessError(1, cmd)
            return types.SimpleNamespace(returncode=1, stdout="no")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return types.SimpleNamespace(returncode=0, stdout="")

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises((RuntimeError, subprocess.CalledProcessError)):
        build.build()
    assert (tmp_path / "LIB").read_text() == (tmp_path / "CALLER").read_text() == "old"


def test_a_missing_extension_says_how_to_build_it(monkeypatch):
    import sys

    import gated_delta_rule_35_amd
    monkeypatch.setitem(sys.modules, "gated_delta_rule_35_amd._kda_py", None)   # its import fails
    monkeypatch.delattr(gated_delta_rule_35_amd, "_kda_py", raising=False)
    with pytest.raises(ImportError, match="build.py"):
        binding._load_caller()
