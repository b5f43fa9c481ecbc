"""What the build makes and when: the library needs no torch, the marshalling module
follows the torch it was built against."""
import os

import pytest
import torch

from parameterized_local_linear_b200 import binding, build


@pytest.fixture
def fakes(tmp_path, monkeypatch):
    """Targets in an empty folder and a subprocess.run that only writes them."""
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libparallax.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    ran = []

    def run(cmd, check):
        ran.append(os.path.basename(cmd[0]))
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            for a in cmd:
                if a.startswith("-DPLX_TORCH_VERSION="):
                    f.write(b"built for torch " + a.split('"')[1].encode() + b"\0")

    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_version_is_torchs():
    assert build.torch_version() == torch.__version__


def test_the_library_builds_without_torch(fakes, monkeypatch):
    monkeypatch.setattr(build, "torch_version", lambda: None)
    assert not build.up_to_date()
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert fakes == ["nvcc"] and not os.path.exists(build.MARSHAL)
    assert build.up_to_date()
    build.build()
    assert fakes == ["nvcc"]


def test_the_module_is_built_again_for_another_torch(fakes, monkeypatch):
    build.build()
    assert fakes == ["nvcc", "g++"] and build.up_to_date()
    monkeypatch.setattr(build, "torch_version", lambda: "9.9.9")
    assert not build.up_to_date()
    build.build()
    assert fakes == ["nvcc", "g++", "g++"] and build.up_to_date()
    build.build(force=True)
    assert fakes[3:] == ["nvcc", "g++"]


def test_a_module_for_another_torch_is_refused(monkeypatch):
    build.build()
    assert binding._marshal().built_for == f"built for torch {torch.__version__}"
    monkeypatch.setattr(binding, "_marshal_module", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError):
        binding._marshal()
