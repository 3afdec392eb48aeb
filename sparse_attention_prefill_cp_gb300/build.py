"""Build libdsa_cp.so in-tree for sm_103a with nvcc (no cmake), and the Python
binding of the calls of a decode step (csrc/binding.cpp) with g++.

Every csrc/*.cu compiles to an object in parallel, then nvcc links the
shared library next to this file, and g++ the binding against it.  Objects go to ``_build/`` at the repo
root (git-ignored).  ``python -m sparse_attention_prefill_cp_gb300.build``
runs it from the command line.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libdsa_cp.so")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")] + ARCH


# Per-source ptxas settings, measured: the attention kernel's pipelined loop
# runs ~1 % faster with ptxas -O1 than with the default -O3 (same registers);
# with -O3 the few-heads attention over the 4-bit cache spills (32 heads: 89
# against 78 us for 152 queries), and the join of its parts moves each load to
# its use instead of keeping them in flight.
SOURCE_FLAGS = {"sparse_attn.cu": ["-Xptxas", "-O1"], "sparse_attn_int4_few.cu": ["-Xptxas", "-O1"],
                "sparse_attn_int4_join.cu": ["-Xptxas", "-O1"]}


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa_cp.so")
    return path


def cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def binding_commands(src: str, obj: str, target: str) -> tuple[list, list]:
    """The compiler's and the linker's command of the Python binding."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    gxx = shutil.which("g++") or "g++"
    include = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda_home(), "include")]
    compile_cmd = [gxx, "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-c", src, "-o", obj] + \
        ["-I" + d for d in include]
    link_cmd = [gxx, "-shared", "-o", target, obj, "-L" + PKG_DIR, "-l:" + os.path.basename(LIB_PATH),
                "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
                "-lc10_cuda"]
    return compile_cmd, link_cmd


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    """Compile (when sources changed) and return the path of libdsa_cp.so."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc()] + NVCC_FLAGS + SOURCE_FLAGS.get(os.path.basename(src), []) + list(extra_flags) + \
                ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    src = os.path.join(CSRC, "binding.cpp")
    binding_obj, tmp_binding = os.path.join(BUILD_DIR, "binding.o"), BINDING_PATH + ".tmp"
    compile_binding, link_binding = binding_commands(src, binding_obj, tmp_binding)
    if force or _stale(binding_obj, [src] + headers):
        if verbose:
            print(" ".join(compile_binding), flush=True)
        procs.append((src, subprocess.Popen(compile_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), flush=True)
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"the compiler failed:\n{msg}")
    if force or procs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("nvcc link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, LIB_PATH)
    if force or procs or _stale(BINDING_PATH, [binding_obj, LIB_PATH]):
        if verbose:
            print(" ".join(link_binding), flush=True)
        r = subprocess.run(link_binding, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("linking the binding failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp_binding, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
