"""Build ``libkda.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled in parallel to an object in
``_build/`` and the objects are linked into ``libkda.so`` next to this file.
The same sources compiled with ``-DKDA_FAULT_INJECTION`` give
``libkda_faultinj.so``, a test-only copy of the library whose
``kda_test_force_timeout`` makes the prefill's bounded device wait give up on
purpose (the tests use it to check the timeout path); both are built in one
parallel pass, and with them ``_kda_torch-<torch version><ABI of the
interpreter>.so``: the calls of ``csrc/py_mla.cpp``, compiled by the host compiler
against the headers of the torch and the Python that run.  The libraries do not
wait for it: where it fails to compile they are linked before the error is
raised.  Usage: ``python -m serving_kda_chunked_gb300.build [--force]``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
FAULTINJ_LIB = os.path.join(HERE, "libkda_faultinj.so")
CALLS_SRC = os.path.join(CSRC, "py_mla.cpp")
CALLS_LIB = os.path.join(HERE, "_kda_torch-%s%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX")))
VARIANTS = ((LIB, "", []), (FAULTINJ_LIB, "faultinj", ["-DKDA_FAULT_INJECTION"]))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")
    return p


def _calls_command(out: str) -> list[str]:
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = [shutil.which(os.environ.get("CXX", "g++")) or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(),
           "-I", INCLUDE]
    for inc in (sysconfig.get_paths()["include"], os.path.join(tdir, "include"),
                os.path.join(cuda, "include")):
        cmd += ["-isystem", inc]
    return cmd + [CALLS_SRC, "-o", out, "-L" + os.path.join(tdir, "lib"), "-ltorch_python",
                  "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _fresh(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _libs_fresh() -> bool:
    return all(_fresh(lib, _deps()) for lib, _, _ in VARIANTS)


def _calls_fresh() -> bool:
    return _fresh(CALLS_LIB, [CALLS_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    return _libs_fresh() and _calls_fresh()


class _Failed:
    """A compiler that could not be started."""
    returncode = 1

    def __init__(self, error):
        self.text = str(error).encode()

    def communicate(self):
        return self.text, None


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        return _Failed(e)


def _finish(procs, verbose) -> list:
    """Waits for the compilers; (source, output) of those that failed."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    return failed


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    libs, calls = force or not _libs_fresh(), force or not _calls_fresh()
    if not (libs or calls):
        return LIB
    cc = nvcc()
    calls_procs, procs, links = [], [], []
    calls_tmp = CALLS_LIB + ".tmp.%d" % os.getpid()
    if calls:
        calls_procs.append((CALLS_SRC, _start(_calls_command(calls_tmp), verbose)))
    for lib, sub, vflags in VARIANTS if libs else ():
        bdir = os.path.join(BUILD, sub) if sub else BUILD
        os.makedirs(bdir, exist_ok=True)
        flags = NVCC_FLAGS + vflags + list(extra_flags or [])
        objs = []
        for src in sources():
            obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
            objs.append(obj)
            procs.append((src, _start([cc, *ARCH, *flags, "-c", src, "-o", obj], verbose)))
        links.append((lib, objs))
    failed = _finish(procs, verbose)
    if not failed:
        for lib, objs in links:
            tmp = lib + ".tmp.%d" % os.getpid()
            subprocess.run([cc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp], check=True)
            os.replace(tmp, lib)
    calls_failed = _finish(calls_procs, verbose)
    if calls and not calls_failed:
        os.replace(calls_tmp, CALLS_LIB)
    if failed or calls_failed:
        msg = "\n".join("%s:\n%s" % (s, t) for s, t in failed + calls_failed)
        raise RuntimeError("compiling failed:\n" + msg)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
