"""The build's own decisions, without building: where CUDA's headers are."""
import os
import shutil

import pytest

from schnet_gnn_molecular_b200 import build


@pytest.mark.parametrize("how", ["name on PATH", "full path", "link elsewhere"])
def test_cuda_headers_are_found_from_nvcc(monkeypatch, tmp_path, how):
    real = shutil.which(build.NVCC)
    if real is None:
        pytest.skip("no nvcc")
    if how == "name on PATH":
        monkeypatch.setenv("PATH", os.path.dirname(real) + os.pathsep + os.environ["PATH"])
        monkeypatch.setattr(build, "NVCC", "nvcc")
    elif how == "link elsewhere":
        os.symlink(real, tmp_path / "nvcc")
        monkeypatch.setattr(build, "NVCC", str(tmp_path / "nvcc"))
    monkeypatch.delenv("CUDA_HOME", raising=False)
    monkeypatch.setattr(build, "CUDA_DEFAULT", str(tmp_path / "none"))
    assert os.path.exists(os.path.join(build.cuda_include(), "cuda_runtime_api.h"))


def test_missing_cuda_headers_are_reported(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setattr(build, "CUDA_DEFAULT", str(tmp_path / "none"))
    monkeypatch.setenv("CUDA_HOME", str(tmp_path))
    with pytest.raises(RuntimeError, match="cuda_runtime_api.h"):
        build.cuda_include()
