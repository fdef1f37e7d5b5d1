"""The build's own decisions, without building: where CUDA's headers are."""
import importlib.metadata
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


@pytest.fixture
def calls(monkeypatch, tmp_path):
    """What build() would do, with a library and a binding newer than their sources."""
    done = []
    for name, attr in (("lib.so", "LIB"), ("binding.so", "BINDING")):
        (tmp_path / name).write_bytes(b"")
        monkeypatch.setattr(build, attr, str(tmp_path / name))
    monkeypatch.setattr(build, "_build_library", lambda verbose, extra: done.append("library"))
    monkeypatch.setattr(build, "_build_binding", lambda verbose: done.append("binding"))
    return done


def test_a_binding_of_another_pytorch_is_stale(monkeypatch, calls):
    build.build()
    assert calls == ["binding"]                   # built for nobody knows what
    build.build()
    assert calls == ["binding"]
    monkeypatch.setattr(build, "built_for", lambda: "torch 0.1 cpython-27")
    build.build()
    assert calls == ["binding", "binding"]
    build.build()
    assert calls == ["binding", "binding"]


def test_the_library_alone_needs_no_pytorch(monkeypatch, calls):
    def gone():
        raise importlib.metadata.PackageNotFoundError("torch")
    build.build(binding=False)
    assert calls == []
    monkeypatch.setattr(build, "built_for", gone)
    build.build()                                 # no PyTorch: nothing to bind to
    build.build(force=True)
    assert calls == ["library"]
