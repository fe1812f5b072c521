"""Build libspec_verify.so in-tree with nvcc for sm_103a.

Two translation units (the verify step, the paged cache operators), one
-gencode, no cmake (about a minute of nvcc).  The checked variant,
libspec_verify_checked.so, is the same source compiled with -DSV_CHECKED: every
global index that a verify or paged kernel forms is tested against its buffer
before the access (a failure sets SV_DEV_OUT_OF_BOUNDS instead of faulting);
the tests run it on small and odd shapes.  All compile in parallel.
``python -m speculative_decoding_verification_25_gb300.build``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libspec_verify.so")
LIB_CHECKED = os.path.join(PKG, "libspec_verify_checked.so")
SRCS = [os.path.join(PKG, "csrc", f) for f in ("spec_verify.cu", "spec_paged.cu")]
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(lib: str) -> bool:
    srcs = [os.path.join(PKG, "csrc", f) for f in os.listdir(os.path.join(PKG, "csrc"))]
    srcs.append(os.path.join(INCLUDE, "spec_verify.h"))
    return (not os.path.exists(lib)
            or os.path.getmtime(lib) < max(os.path.getmtime(s) for s in srcs))


def _object(lib: str, src: str) -> str:
    return os.path.join(PKG, "build", os.path.basename(lib)[3:-3] + "." + os.path.basename(src) + ".o")


def _cmd(lib: str, src: str, checked: bool, verbose: bool):
    cmd = [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-c", "-Xcompiler", "-fPIC",
           "-I" + INCLUDE, "-o", _object(lib, src), src]
    if checked:
        cmd.insert(1, "-DSV_CHECKED")
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def _link_cmd(lib: str):
    return [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", lib + ".tmp",
            *(_object(lib, src) for src in SRCS)]


def _run_all(cmds, verbose: bool):
    """Runs the commands at once; raises with the output of those that failed."""
    procs = [(cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
             for cmd in cmds]
    errors = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append("nvcc failed:\n" + " ".join(cmd) + "\n" + out)
        elif verbose:
            sys.stderr.write(out)
    if errors:
        raise RuntimeError("\n".join(errors))


def build(verbose: bool = False, force: bool = False, checked: bool = True) -> str:
    """Compile the library (and, with ``checked``, its checked variant)
    when a source is newer than it or ``force``; returns the library path."""
    jobs = [(LIB, False)] + ([(LIB_CHECKED, True)] if checked else [])
    jobs = [(lib, chk) for lib, chk in jobs if force or _stale(lib)]
    os.makedirs(os.path.join(PKG, "build"), exist_ok=True)
    _run_all([_cmd(lib, src, chk, verbose) for lib, chk in jobs for src in SRCS], verbose)
    _run_all([_link_cmd(lib) for lib, _ in jobs], verbose)
    for lib, _ in jobs:
        os.replace(lib + ".tmp", lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force=True))
