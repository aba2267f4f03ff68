"""Builds libengram.so in-tree with nvcc for sm_103a (two translation units, compiled side by side) and, with
the host compiler, the binding's marshalling module for the decode-step calls (against torch's headers)."""

import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
SRC_DIR = os.path.join(HERE, "csrc")
MAIN_SRCS = [os.path.join(SRC_DIR, f) for f in ("engram_core.cu", "attention.cu")]
LIB_PATH = os.path.join(HERE, "libengram.so")
OBJ_DIR = os.path.join(HERE, "_build")
STEP_SRC = os.path.join(SRC_DIR, "step_binding.cpp")
STEP_PATH = os.path.join(HERE, "_step.so")
STEP_STAMP = os.path.join(OBJ_DIR, "_step.torch")  # the torch and Python that it was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def sources():
    out = []
    for d in (SRC_DIR, os.path.join(os.path.dirname(HERE), "include")):
        for f in sorted(os.listdir(d)):
            if f.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(d, f))
    return out


def _stale(path, srcs):
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in srcs)


def _against():
    import torch

    return f"{torch.__version__} {sysconfig.get_config_var('EXT_SUFFIX')}"


def step_stale():
    """Whether the binding module is older than its sources or was built against another torch or Python (it uses
    torch's C++ interface, which changes from one version to the next)."""
    if _stale(STEP_PATH, [STEP_SRC, os.path.join(os.path.dirname(HERE), "include", "engram.h")]):
        return True
    if not os.path.exists(STEP_STAMP):
        return True
    with open(STEP_STAMP, encoding="utf-8") as f:
        return f.read() != _against()


def step_cmd():
    import torch

    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{d}" for d in include], "-o", STEP_PATH, STEP_SRC, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", f"-Wl,-rpath,{lib}"]


def compile_cmd(src, obj, extra=()):
    return ["nvcc", *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", *extra, "-c", "-o", obj, src]


def link_cmd(objs, out=LIB_PATH):
    return ["nvcc", *ARCH, "-shared", "-o", out, *objs]


def build(force=False, verbose=False):
    """Compile what is older than its sources; returns the library's path."""
    cmds, objs, step = [], [], force or step_stale()
    if force or _stale(LIB_PATH, sources()):
        os.makedirs(OBJ_DIR, exist_ok=True)
        objs = [os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(s))[0] + ".o") for s in MAIN_SRCS]
        cmds += [compile_cmd(s, o) for s, o in zip(MAIN_SRCS, objs)]
    if step:
        os.makedirs(OBJ_DIR, exist_ok=True)
        cmds.append(step_cmd())
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd))
    procs = [subprocess.Popen(cmd) for cmd in cmds]
    codes = [p.wait() for p in procs]
    for cmd, code in zip(cmds, codes):
        if code:
            raise subprocess.CalledProcessError(code, cmd)
    if step:
        with open(STEP_STAMP, "w", encoding="utf-8") as f:
            f.write(_against())
    if objs:
        subprocess.check_call(link_cmd(objs))
    return LIB_PATH
