"""Build libdsa_cp.so in-tree for sm_103a with nvcc (no cmake), and the Python
binding of the calls of a decode step (csrc/binding.cpp) with g++.

Every csrc/*.cu compiles to an object in parallel, then nvcc links the
shared library next to this file, and g++ the binding against it.  The library
needs nvcc alone: it is there whether or not the binding, which needs the
headers of torch and of Python, can be built.  Objects go to ``_build/`` at
the repo root (git-ignored).  ``python -m sparse_attention_prefill_cp_gb300.build``
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


def binding_tag() -> str:
    """The Python and the torch that a binding is for; both are in its file's name, so that after a change of either it is
    built again instead of loaded."""
    import torch
    return f"{sys.implementation.cache_tag}-torch{torch.__version__}"


def binding_path() -> str:
    return os.path.join(PKG_DIR, f"_binding.{binding_tag()}.so")


def binding_object() -> str:
    return os.path.join(BUILD_DIR, f"binding.{binding_tag()}.o")


def binding_commands(src: str, obj: str, target: str) -> tuple[list, list]:
    """The compiler's and the linker's command of the Python binding."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    gxx = shutil.which("g++") or "g++"
    include = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda_home(), "include")]
    compile_cmd = [gxx, "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-c", src, "-o", obj] + \
        ["-I" + d for d in include]
    link_cmd = [gxx, "-shared", "-o", target, obj, "-L" + os.path.dirname(LIB_PATH), "-l:" + os.path.basename(LIB_PATH),
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


def _headers() -> list:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _start(cmd: list, verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs: list, verbose: bool) -> None:
    """Wait for the compilers of (source, process); raise what the failed ones said."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), flush=True)
    if failed:
        raise RuntimeError("the compiler failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed))


def _link(cmd: list, tmp: str, target: str, verbose: bool) -> None:
    _finish([(target, _start(cmd, verbose))], verbose)
    os.replace(tmp, target)


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    """Compile (when sources changed) and return the path of libdsa_cp.so; with
    torch there, the binding too."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = _headers()
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            procs.append((src, _start([nvcc()] + NVCC_FLAGS + SOURCE_FLAGS.get(os.path.basename(src), []) +
                                      list(extra_flags) + ["-c", src, "-o", obj], verbose)))
    binding, fault = None, None
    try:
        if importlib.util.find_spec("torch") is not None:
            binding = compile_binding(verbose, force)
    except Exception as e:  # raised when the library is there
        fault = e
    try:
        _finish(procs, verbose)
        if force or procs or _stale(LIB_PATH, objs):
            tmp = LIB_PATH + ".tmp"
            _link([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs, tmp, LIB_PATH, verbose)
    except BaseException:
        for _, p in binding or []:
            p.communicate()
        raise
    if fault is not None:
        raise fault
    if binding is not None:
        link_binding(binding, verbose, force)
    return LIB_PATH


def compile_binding(verbose: bool = False, force: bool = False) -> list:
    """Start the binding's compiler where its object is not up to date: [(source, process)] or []."""
    src = os.path.join(CSRC, "binding.cpp")
    if not (force or _stale(binding_object(), [src] + _headers())):
        return []
    return [(src, _start(binding_commands(src, binding_object(), "")[0], verbose))]


def link_binding(compiling: list, verbose: bool = False, force: bool = False) -> str:
    """Wait for the binding's compiler and link the binding against the library as it is."""
    _finish(compiling, verbose)
    target, obj = binding_path(), binding_object()
    if force or compiling or _stale(target, [obj]):
        tmp = target + ".tmp"
        _link(binding_commands("", obj, tmp)[1], tmp, target, verbose)
    return target


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """The binding alone.  The library is left as it is: a process that has loaded it would load a rebuilt one beside it,
    with an error record of its own."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    return link_binding(compile_binding(verbose, force), verbose, force)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
