"""What the build needs and when it is up to date (no compiler runs here)."""
import os
import subprocess
import sys

import pytest

from audio_encoder_b200 import build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Stands in for the compilers: records their commands, writes what they
    would, into a folder of its own; `missing` ones are not found."""
    class Ran(list):
        missing = ()

        def run(self, cmd, check):
            assert check
            self.append(os.path.basename(cmd[0]))
            if self[-1] in self.missing:
                raise FileNotFoundError(cmd[0])
            open(cmd[cmd.index("-o") + 1], "w").close()

    ran = Ran()
    monkeypatch.setattr(subprocess, "run", ran.run)
    for name in ("LIB", "PYCALLS_LIB"):
        if hasattr(build, name):
            monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    return ran


def test_the_library_builds_without_pytorch(monkeypatch, compilers, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert compilers == ["nvcc"] and os.path.exists(build.LIB)
    assert "PyTorch" in capsys.readouterr().err


def test_the_python_side_fails_after_the_library_and_with_an_error_of_its_own(monkeypatch, compilers):
    pytest.importorskip("torch")
    monkeypatch.delenv("CXX", raising=False)
    compilers.missing = ("g++",)
    with pytest.raises(build.PycallsError, match="is built"):
        build.build()
    assert compilers == ["nvcc", "g++"] and os.path.exists(build.LIB)
    compilers.missing = ("nvcc",)  # the library is there, so only the other is built
    assert build.build() == build.LIB and compilers[2:] == ["g++"]
    assert build.build() == build.LIB and len(compilers) == 3  # nothing to do


def test_another_pytorch_or_python_needs_another_python_side(monkeypatch, compilers):
    # it is bound to the ABI of both
    torch = pytest.importorskip("torch")
    build.build()
    monkeypatch.setattr(torch, "__version__", "99.1")
    build.build()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-999")
    build.build()
    assert [c for c in compilers if c != "nvcc"] == compilers[1:] and len(compilers) == 4
    files = [f for f in os.listdir(build.HERE) if f.startswith("_pycalls")]
    assert len(files) == 3 and any("99.1" in f and "cpython-999" in f for f in files)
    monkeypatch.setattr(torch, "__version__", "99.2")
    from audio_encoder_b200 import binding
    monkeypatch.setattr(binding, "_pycalls", None)
    with pytest.raises(ImportError, match="99.2"):
        binding.pycalls()


def test_the_library_alone(compilers):
    assert build.build_library() == build.LIB and compilers == ["nvcc"]
