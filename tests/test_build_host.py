"""The build's parts stand by themselves: the CUDA library needs no torch, and
the compiled calls belong to one interpreter and one torch (no GPU needed)."""
import os
import sysconfig

import pytest
import torch

from serving_kda_chunked_gb300 import build as kbuild


def test_calls_are_kept_per_interpreter_and_torch():
    name = os.path.basename(kbuild.CALLS_LIB)
    assert torch.__version__ in name
    assert name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build over one empty kernel, in a folder of its own."""
    src = tmp_path / "small.cu"
    src.write_text("__global__ void k() {}\nextern \"C\" int small_answer() { return 42; }\n")
    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(kbuild, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(kbuild, "CALLS_LIB", str(tmp_path / "calls.so"))
    monkeypatch.setattr(kbuild, "VARIANTS", ((str(tmp_path / "libkda.so"), "", []),))
    monkeypatch.setattr(kbuild, "sources", lambda: [str(src)])
    return tmp_path


def test_library_is_linked_where_the_calls_do_not_compile(small, monkeypatch):
    compiler = small / "no-compiler"
    compiler.write_text("#!/bin/sh\necho no such header >&2\nexit 1\n")
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    with pytest.raises(RuntimeError, match="py_mla.cpp(.|\n)*no such header"):
        kbuild.build(force=True)
    assert (small / "libkda.so").exists() and not (small / "calls.so").exists()
    # nor where there is no compiler to start
    (small / "libkda.so").unlink()
    real_popen = kbuild.subprocess.Popen

    def popen(cmd, **kw):
        if kbuild.CALLS_SRC in cmd:
            raise FileNotFoundError("no such compiler: " + cmd[0])
        return real_popen(cmd, **kw)

    monkeypatch.setattr(kbuild.subprocess, "Popen", popen)
    with pytest.raises(RuntimeError, match="py_mla.cpp(.|\n)*no such compiler"):
        kbuild.build(force=True)
    assert (small / "libkda.so").exists()


def test_one_part_does_not_make_the_other_stale(small, monkeypatch):
    compiler = small / "quick-compiler"
    compiler.write_text("#!/bin/sh\nwhile [ \"$1\" != -o ]; do shift; done\necho calls > \"$2\"\n")
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    kbuild.build()
    assert kbuild.up_to_date()
    linked = os.path.getmtime(small / "libkda.so")
    (small / "calls.so").unlink()
    assert not kbuild.up_to_date()
    kbuild.build()
    assert kbuild.up_to_date() and os.path.getmtime(small / "libkda.so") == linked
