"""The build script with stand-in compilers: what is built when a part cannot be, and when the
binding is built again."""
import os
import sysconfig

import pytest

from structured_sparse_gemm_compress_b200 import build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """Outputs under tmp_path; compilers that write their output file and log the call."""
    log = tmp_path / "calls"
    log.write_text("")

    def compiler(name, works=True):
        path = tmp_path / name
        path.write_text(f"#!/bin/sh\necho {name} >> {log}\n" + (
            'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then : > "$2"; fi; shift; done\n' if works else "exit 1\n"))
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "_compile", lambda src, force, extra, objdir: _object(objdir, src))
    monkeypatch.setattr(build, "NVCC", compiler("nvcc"))
    monkeypatch.setattr(build, "CXX", compiler("cxx"))
    return compiler, lambda: log.read_text().split()


def _object(objdir, src):
    path = os.path.join(objdir, src + ".o")
    open(path, "w").close()
    return path


def test_library_is_built_without_a_cxx_compiler(sandbox, monkeypatch):
    compiler, _ = sandbox
    monkeypatch.setattr(build, "CXX", compiler("broken", works=False))
    with pytest.raises(RuntimeError, match="is built, but not the Python binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_library_is_built_without_a_cxx_program(sandbox, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CXX", str(tmp_path / "absent"))
    with pytest.raises(RuntimeError, match="is built, but not the Python binding"):
        build.build()
    assert os.path.exists(build.LIB)


def test_binding_is_built_again_for_another_python(sandbox, monkeypatch):
    _, calls = sandbox
    build.build()
    assert os.path.exists(build.LIB) and calls().count("cxx") == 1
    build.build()
    assert calls().count("cxx") == 1
    var = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else var(name))
    build.build()
    build.build()
    assert calls().count("cxx") == 2
