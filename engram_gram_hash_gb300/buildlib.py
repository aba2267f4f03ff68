"""Builds libengram.so in-tree with nvcc for sm_103a (two translation units, compiled side by side)."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
SRC_DIR = os.path.join(HERE, "csrc")
MAIN_SRCS = [os.path.join(SRC_DIR, f) for f in ("engram_core.cu", "attention.cu")]
LIB_PATH = os.path.join(HERE, "libengram.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def sources():
    out = []
    for d in (SRC_DIR, os.path.join(os.path.dirname(HERE), "include")):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(d, f))
    return out


def compile_cmd(src, obj, extra=()):
    return ["nvcc", *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", *extra, "-c", "-o", obj, src]


def link_cmd(objs, out=LIB_PATH):
    return ["nvcc", *ARCH, "-shared", "-o", out, *objs]


def build(force=False, verbose=False):
    """Compile if any source is newer than the library; returns its path."""
    stale = force or not os.path.exists(LIB_PATH)
    if not stale:
        t = os.path.getmtime(LIB_PATH)
        stale = any(os.path.getmtime(s) > t for s in sources())
    if stale:
        objs = [os.path.splitext(s)[0] + ".o" for s in MAIN_SRCS]
        cmds = [compile_cmd(s, o) for s, o in zip(MAIN_SRCS, objs)]
        if verbose:
            for cmd in cmds:
                print(" ".join(cmd))
        procs = [subprocess.Popen(cmd) for cmd in cmds]
        codes = [p.wait() for p in procs]
        for cmd, code in zip(cmds, codes):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.check_call(link_cmd(objs))
    return LIB_PATH
