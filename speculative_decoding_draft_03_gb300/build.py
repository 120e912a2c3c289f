"""Build the CUDA library ``libdspark.so`` in-tree for sm_103a (GB300).

Each translation unit is compiled in parallel with nvcc, then linked into one shared
library with the shared CUDA runtime (the same ``libcudart.so.13`` PyTorch loads).  Beside it
stands ``_marshal.so``, the host-side marshalling of the serving calls, compiled with g++ against
PyTorch's headers and linked to the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libdspark.so")
MARSHAL = os.path.join(BUILD, "_marshal.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills", "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _marshal_commands(obj: str, target: str):
    """Compiling and linking the marshalling module against the PyTorch that imports it."""
    import torch
    root = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
    link = [cxx, "-shared", "-o", target, obj, "-L", os.path.dirname(LIB), "-ldspark", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    return compile_, link


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _holds(path, text) -> bool:
    if not os.path.exists(path):
        return False
    with open(path) as f:
        return f.read() == text


def build(verbose: bool = False, force: bool = False, extra_flags=(), build_dir: str = BUILD) -> str:
    """Compile every csrc/*.cu and link libdspark.so in `build_dir` (the package's _build by
    default, where the marshalling module stands too; tests build variants with extra -D flags
    into their own directories)."""
    os.makedirs(build_dir, exist_ok=True)
    lib = os.path.join(build_dir, "libdspark.so")
    nvcc = _nvcc()
    srcs = _sources()
    hdrs = _headers()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(build_dir, os.path.basename(s).replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    marshal = build_dir == BUILD
    if marshal:
        # (named after the PyTorch that it is compiled against: another one compiles its own)
        import torch
        obj = os.path.join(build_dir, f"marshal-{torch.__version__}.o")
        compile_, link = _marshal_commands(obj, MARSHAL + f".tmp{os.getpid()}")
        if force or _stale(obj, [os.path.join(CSRC, "marshal.cpp")] + hdrs):
            jobs.append(compile_)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compilation failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return r

    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
        os.replace(tmp, lib)
    stamp = os.path.join(build_dir, "marshal.stamp")
    if marshal and (force or _stale(MARSHAL, [obj, lib]) or not _holds(stamp, torch.__version__)):
        run(link)
        os.replace(MARSHAL + f".tmp{os.getpid()}", MARSHAL)
        with open(stamp, "w") as f:
            f.write(torch.__version__)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
