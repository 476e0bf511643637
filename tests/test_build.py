"""The build finds CUDA's headers from nvcc however it is named, and a binding that
cannot be compiled does not keep the library from being installed."""
import os
import subprocess

import pytest

from w4a4_post_quantization_b200 import build as b


def headers_found(command):
    return [d for flag, d in zip(command, command[1:]) if flag == "-isystem"
            and os.path.exists(os.path.join(d, "cuda_runtime_api.h"))]


def test_a_bare_compiler_name(monkeypatch):
    assert headers_found(b._binding_command())
    bin_dir = os.path.dirname(b.NVCC)
    monkeypatch.setenv("PATH", bin_dir + os.pathsep + os.environ["PATH"])
    monkeypatch.setattr(b, "NVCC", "nvcc")
    assert headers_found(b._binding_command())


def test_a_link_to_the_compiler(monkeypatch, tmp_path):
    (tmp_path / "nvcc").symlink_to(b.NVCC)
    monkeypatch.setattr(b, "NVCC", str(tmp_path / "nvcc"))
    assert headers_found(b._binding_command())


@pytest.fixture
def small(monkeypatch, tmp_path):
    """A library of one function and a binding, both built under tmp_path."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libone.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    return tmp_path


def missing():
    raise ImportError("torch")


@pytest.mark.parametrize("command,error", [(lambda: ["false"], subprocess.CalledProcessError), (missing, ImportError),
                                           (lambda: ["/no/such/compiler"], OSError)])
def test_the_library_is_there_without_its_binding(small, monkeypatch, command, error):
    monkeypatch.setattr(b, "_binding_command", command)
    with pytest.raises(error):
        b.build(force=True)
    assert (small / "libone.so").exists() and not (small / "binding.so").exists()


def test_a_library_that_does_not_compile_is_not_installed(small, monkeypatch):
    (small / "one.cu").write_text("not a program\n")
    monkeypatch.setattr(b, "_binding_command", lambda: ["cp", str(small / "one.cu"), b.BINDING + ".tmp"])
    with pytest.raises(subprocess.CalledProcessError):
        b.build(force=True)
    assert not (small / "libone.so").exists()
