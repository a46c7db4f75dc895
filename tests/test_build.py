"""The build's host logic, with the compilers replaced (nothing is compiled here)."""
import os
import subprocess

import pytest

from bit_diffusion_transformer_b200 import build as b


class Jobs:
    """Stands for the compiler processes: writes each command's -o file, or fails the named source."""

    def __init__(self, monkeypatch, fails=None):
        self.commands, self.fails = [], fails
        monkeypatch.setattr(b.subprocess, "Popen", self.popen)
        monkeypatch.setattr(b.subprocess, "check_call", self.check_call)

    def run(self, cmd):
        self.commands.append(cmd)
        if self.fails and any(self.fails in part for part in cmd):
            return 1
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return 0

    def popen(self, cmd, **kw):
        code = self.run(cmd)
        return type("Job", (), {"wait": lambda self: code})()

    def check_call(self, cmd, **kw):
        if self.run(cmd):
            raise subprocess.CalledProcessError(1, cmd)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Targets in an empty folder."""
    monkeypatch.setattr(b, "SO", str(tmp_path / "libopq.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "_fp8.so"))
    return tmp_path


def cuda_toolkit(path):
    (path / "bin").mkdir(parents=True)
    (path / "include").mkdir()
    (path / "include" / "cuda_runtime_api.h").write_text("")
    nvcc = path / "bin" / "nvcc"
    nvcc.write_text("#!/bin/sh\n")
    nvcc.chmod(0o755)
    return nvcc


@pytest.mark.parametrize("link", [False, True])
def test_cuda_headers_with_nvcc_on_the_path(tree, monkeypatch, link):
    nvcc = cuda_toolkit(tree / "toolkit")
    folder = nvcc.parent
    if link:                                   # as /usr/bin/nvcc may point into the toolkit
        folder = tree / "somewhere" / "bin"
        folder.mkdir(parents=True)
        (folder / "nvcc").symlink_to(nvcc)
    monkeypatch.setenv("PATH", str(folder) + os.pathsep + os.environ["PATH"])
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    jobs = Jobs(monkeypatch)
    b.build()
    ext = next(c for c in jobs.commands if any(part.endswith(b.EXT_SOURCE) for part in c))
    assert os.path.realpath(tree / "toolkit" / "include") in [os.path.realpath(p) for p in ext]


@pytest.mark.parametrize("how", ["compiler fails", "no CUDA headers"])
def test_library_is_linked_where_the_binding_cannot_be_built(tree, monkeypatch, how):
    Jobs(monkeypatch, fails=b.EXT_SOURCE if how == "compiler fails" else None)
    if how == "no CUDA headers":
        monkeypatch.setattr(b, "_nvcc", lambda: str(tree / "toolkit" / "bin" / "nvcc"))
    with pytest.raises(subprocess.CalledProcessError if how == "compiler fails" else FileNotFoundError):
        b.build()
    assert os.path.exists(b.SO) and not os.path.exists(b.EXT)
    assert sorted(os.listdir(tree)) == ["libopq.so"]


def test_a_failed_kernel_file_leaves_the_old_library(tree, monkeypatch):
    (tree / "libopq.so").write_text("old")
    os.utime(tree / "libopq.so", (1, 1))
    Jobs(monkeypatch, fails="opq_capi.cu")
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert (tree / "libopq.so").read_text() == "old" and sorted(os.listdir(tree)) == ["libopq.so"]


def test_binding_is_built_again_for_another_torch(tree, monkeypatch):
    jobs = Jobs(monkeypatch)
    b.build()
    n = len(jobs.commands)
    b.build()
    assert len(jobs.commands) == n             # nothing to do
    import torch
    monkeypatch.setattr(torch, "__version__", "99.1.0+cu999")
    b.build()
    again = jobs.commands[n:]
    assert again and all("nvcc" not in c[0] for c in again)     # the binding alone
    b.build()
    assert len(jobs.commands) == n + len(again)


def test_binding_of_another_torch_is_refused(monkeypatch):
    import torch

    from bit_diffusion_transformer_b200 import build, fp8
    build.build()
    monkeypatch.setattr(fp8, "_ext", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "99.1.0+cu999")
        with pytest.raises(ImportError, match="99.1.0"):
            fp8._load()
    assert fp8._load() is not None


def test_binding_takes_every_build_of_its_torch(monkeypatch):
    import torch

    from bit_diffusion_transformer_b200 import build, fp8
    build.build()
    number = fp8._load().TORCH_VERSION
    for version, ok in ((number, True), (number + "+cu130", True), (number + "a0+gitabc.nv25", True),
                        (number + "7", False), ("1" + number, False)):
        monkeypatch.setattr(fp8, "_ext", None)
        monkeypatch.setattr(torch, "__version__", version)
        if ok:
            fp8._load()
        else:
            with pytest.raises(ImportError):
                fp8._load()
