"""Build libpararnn.so, libpararnn_lm.so and libpararnn_block.so (HIP, gfx950 only) in-tree with hipcc.

    python -m nonlinear_rnn_solve_amd.build            # build the libraries and their look-back stress variants
    python -m nonlinear_rnn_solve_amd.build --asm      # also keep the gfx950 assembly for inspection

Flags: -O3, --offload-arch=gfx950, the packed-fp32 instructions disabled
(-Xclang -target-feature -Xclang -packed-fp32-ops; hipcc's host pass prints
that it does not know that feature, the device pass honours it), and
-ffp-contract=on: a multiply and an add fuse into an fma only within one source
expression (or where the source calls fmaf), never across statements, so a
computation inlined into two kernels rounds the same way in both.

libpararnn_stress.so is the same source with -DPR_LB_STRESS=1: tiles pause for
pseudo-random times before publishing look-back words, so that scans walk far
back.  Only the tests load it; its results must equal libpararnn.so's bit for bit.

libpararnn_lm.so holds the language-model operators of include/pararnn_lm.h, one source file each, compiled in
parallel and linked; _lm_binding.*.so is its Python binding (host C++ against torch's headers; without torch or g++ it
is left out, with a message, since the C ABI needs neither), and libpararnn_lm_stress.so its look-back stress variant.
libpararnn_block.so and _block_binding.*.so are the same for the block operators of include/pararnn_block.h.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "pararnn.hip")
INC = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpararnn.so")
STRESS_LIB = os.path.join(HERE, "libpararnn_stress.so")
LM_SRCS = [os.path.join(HERE, "csrc", f) for f in ("lm_scan.hip", "lm_norm.hip", "lm_logp.hip")]
LM_LIB = os.path.join(HERE, "libpararnn_lm.so")
LM_STRESS_LIB = os.path.join(HERE, "libpararnn_lm_stress.so")
LM_BINDING_SRC = os.path.join(HERE, "csrc", "lm_binding.cpp")
LM_BINDING = os.path.join(HERE, "_lm_binding" + sysconfig.get_config_var("EXT_SUFFIX"))   # of this interpreter
BLOCK_SRCS = [os.path.join(HERE, "csrc", f) for f in ("block_ssm.hip", "block_conv.hip", "block_ffn.hip", "block_adamw.hip")]
BLOCK_LIB = os.path.join(HERE, "libpararnn_block.so")
BLOCK_BINDING_SRC = os.path.join(HERE, "csrc", "block_binding.cpp")
BLOCK_BINDING = os.path.join(HERE, "_block_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = "gfx950"


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    p = os.path.join(rocm, "bin", "hipcc")
    return p if os.path.exists(p) else "hipcc"


FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-ffp-contract=on",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wall", "-Wno-unused-function", "-I", INC]


def _command(out: str, stress: bool, asm: bool) -> list:
    cmd = [hipcc()] + FLAGS + ["-shared", SRC, "-o", out]
    if stress:
        cmd.insert(1, "-DPR_LB_STRESS=1")
    if asm:
        cmd += ["--save-temps"]
    return cmd


def build(asm: bool = False, verbose: bool = True, stress: bool = True) -> str:
    """Compile libpararnn.so, libpararnn_lm.so, libpararnn_block.so (and, with stress, the stress variants), all in parallel;
    returns the path of libpararnn.so."""
    bindings = _binding_commands()   # before anything is started
    jobs = [(LIB, False)] + ([(STRESS_LIB, True)] if stress else [])
    if asm:
        os.makedirs(os.path.join(ROOT, "_build"), exist_ok=True)
    procs = []
    for lib, st in jobs:
        tmp = lib + ".tmp%d" % os.getpid()
        cmd = _command(tmp, st, asm and not st)
        procs.append((_start(cmd, verbose, os.path.join(ROOT, "_build") if (asm and not st) else HERE), tmp, lib))
    block = _start_objects(verbose, BLOCK_SRCS)
    lm = _start_objects(verbose, LM_SRCS)
    compiling = [_start_binding(b, verbose) for b in bindings]
    lm_stress = _start_objects(verbose, LM_SRCS[:1], "PR_LB_STRESS=1") if stress else []
    failed = _finish(procs, verbose)
    failed += _finish_objects(lm, LM_LIB, verbose)
    if stress:
        failed += _finish_objects(lm_stress, LM_STRESS_LIB, verbose)
    failed += _finish_objects(block, BLOCK_LIB, verbose)
    for b, jobs in zip(bindings, compiling):
        failed += _finish_binding(b, jobs, verbose, not failed)
    if failed:
        raise RuntimeError("hipcc failed: %s" % failed)
    return LIB


def _start(cmd, verbose, cwd=HERE):
    if verbose:
        print("[build]", " ".join(cmd), flush=True)
    return subprocess.Popen(cmd, cwd=cwd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _start_objects(verbose, srcs, define=None):
    """Start compiling a library's sources; objects beside the library until it is linked."""
    jobs = []
    for src in srcs:
        obj = os.path.join(HERE, "%s%s.tmp%d.o" % (os.path.basename(src)[:-4], "_stress" if define else "", os.getpid()))
        cmd = [hipcc()] + FLAGS + (["-D" + define] if define else []) + ["-c", src, "-o", obj]
        jobs.append((_start(cmd, verbose), obj, obj))
    return jobs


def _finish_objects(jobs, lib, verbose):
    failed = _finish(jobs, verbose)
    objs = [obj for _, _, obj in jobs]
    if not failed:
        tmp = lib + ".tmp%d" % os.getpid()
        link = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC"] + objs + ["-o", tmp]
        failed = _finish([(_start(link, verbose), tmp, lib)], verbose)
    for obj in objs:
        if os.path.exists(obj):
            os.remove(obj)
    return failed


def _binding_commands():
    """(object, compile command, link command without its output, binding) of each binding; none where torch or g++ is
    missing."""
    missing = "torch" if importlib.util.find_spec("torch") is None else "g++" if shutil.which("g++") is None else None
    if missing:
        print("[build] %s and %s are left out: no %s (nonlinear_rnn_solve_amd.lm and .block need them, the C ABI does not)"
              % (os.path.basename(LM_BINDING), os.path.basename(BLOCK_BINDING), missing), flush=True)
        return []
    import torch
    from torch.utils.cpp_extension import include_paths
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", "-I", INC]
    for p in include_paths() + [os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", p]
    found = []
    for src, lib, binding in ((LM_BINDING_SRC, "pararnn_lm", LM_BINDING), (BLOCK_BINDING_SRC, "pararnn_block", BLOCK_BINDING)):
        obj = os.path.join(HERE, "%s.tmp%d.o" % (os.path.basename(src)[:-4], os.getpid()))
        link = ["g++", "-shared", obj, "-L", HERE, "-l" + lib, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
                "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
        found.append((obj, cmd + ["-c", src, "-o", obj], link, binding))
    return found


def _start_binding(commands, verbose):
    """Start compiling a binding; its object beside it until it is linked against its library."""
    obj, compile_, _, _ = commands
    return [(_start(compile_, verbose), obj, obj)]


def _finish_binding(commands, jobs, verbose, link):
    failed = _finish(jobs, verbose)
    obj, _, cmd, binding = commands
    tmp = binding + ".tmp%d" % os.getpid()
    if link and not failed:
        failed = _finish([(_start(cmd + ["-o", tmp], verbose), tmp, binding)], verbose)
    if os.path.exists(obj):
        os.remove(obj)
    return failed


def _finish(procs, verbose):
    failed = []
    for p, tmp, lib in procs:
        out, _ = p.communicate()
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
        if out.strip() and verbose:
            print(out)
        if p.returncode != 0:
            failed.append((lib, p.returncode))
        elif tmp != lib:
            os.replace(tmp, lib)
    return failed


if __name__ == "__main__":
    if "--asm" in sys.argv:
        os.makedirs(os.path.join(ROOT, "_work"), exist_ok=True)
    build(asm="--asm" in sys.argv)
