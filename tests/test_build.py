"""The C library's build asks for nvcc alone: no torch with CUDA, no Python headers, no compiler by another name. Commands are
recorded here and not run."""

import os
import subprocess
import types

import pytest

from quantized_linear_layers_block_gb300 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """build() with its products in tmp_path; the list of its commands. One that names a word of `fail` fails."""
    seen, fail = [], []

    def run(cmd, **_):
        seen.append(cmd)
        if any(word in part for word in fail for part in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="planted")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    for name in ("LIB", "TENSORS"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "objects"))
    seen_and_fail = types.SimpleNamespace(seen=seen, fail=fail)
    return seen_and_fail


def fake_torch(monkeypatch, tmp_path, cuda):
    d = tmp_path / "torch"
    for f in ["__init__.py"] + (["lib/libc10_cuda.so", "include/c10/cuda/CUDAGuard.h"] if cuda else ["lib/libc10.so"]):
        (d / f).parent.mkdir(parents=True, exist_ok=True)
        (d / f).touch()
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: types.SimpleNamespace(origin=str(d / "__init__.py")))


def test_torch_without_cuda(commands, monkeypatch, tmp_path):
    fake_torch(monkeypatch, tmp_path, cuda=False)
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)
    n = len(commands.seen)
    assert n == len(build.SOURCES) + 1
    build.build()
    assert len(commands.seen) == n          # and there is nothing left to build


def test_no_torch(commands, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)


def test_no_python_headers(commands, monkeypatch, tmp_path):
    fake_torch(monkeypatch, tmp_path, cuda=True)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)


@pytest.mark.parametrize("word", ["tensors.cpp", "tensors.o"])
def test_an_error_in_the_module_leaves_a_library_and_is_raised_each_time(commands, monkeypatch, tmp_path, word):
    fake_torch(monkeypatch, tmp_path, cuda=True)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    (tmp_path / "Python.h").touch()
    commands.fail.append(word)
    for _ in range(2):
        with pytest.raises(RuntimeError):
            build.build()
        assert os.path.exists(build.LIB) and not os.path.exists(build.TENSORS)
    commands.fail.clear()
    build.build()
    assert os.path.exists(build.TENSORS)
    # the library is built anew, the module is not: what is left of the last one does not count
    build.build(force=True)
    commands.fail.append(word)
    os.utime(build.TENSORS, (1, 1))
    with pytest.raises(RuntimeError):
        build.build()


def test_one_compiler(commands):
    build.build()
    assert {os.path.basename(cmd[0]) for cmd in commands.seen} == {"nvcc"}
