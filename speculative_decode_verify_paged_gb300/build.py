"""Build libspec_attn.so in-tree with nvcc for sm_103a.

Each CUDA translation unit under csrc/ is compiled in parallel into
_build/*.o, then linked into _build/libspec_attn.so (CUDA runtime linked
statically, so the library needs only the driver, and nvcc alone builds it).
Where torch is installed, the native side of the Python binding,
csrc/binding.cpp, then becomes the extension module _build/spec_attn_calls.so,
compiled with torch's headers and linked against that library; it has a stamp
of its own, and its failure leaves the library built.  No cmake.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(BUILD, "libspec_attn.so")
CALLS = os.path.join(BUILD, "spec_attn_calls.so")
BINDING = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
                  [os.path.abspath(__file__)])


def _binding_deps():
    return [BINDING] + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def _same(stamp, text):
    if not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == text


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + list(extra) + ["-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _torch():
    """(folder, version) of torch, found without importing it; None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:      # (a source tree on the path)
        version = "unknown"
    return list(spec.submodule_search_locations)[0], version


def _compile_binding(torch_dir):
    """The extension module's object: C++ against the headers of the running interpreter and torch."""
    torch_include = os.path.join(torch_dir, "include")
    obj = os.path.join(BUILD, "binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-c", "-fPIC", "-O2", "-std=c++17", "-Wall", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", torch_include,
           "-isystem", os.path.join(torch_include, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), BINDING, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def _link_binding(obj, torch_dir):
    """The module finds the library beside it, and torch's libraries where the importing process has loaded them."""
    tmp = CALLS + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, LIB, "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every CUDA source and link the shared library, then the binding's module where torch is installed; return
    the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    # the library is also stale when a source was added or removed since it was linked, the module with another torch
    stamp, listing = os.path.join(BUILD, "sources.txt"), "\n".join(os.path.basename(s) for s in srcs)
    lib_due = bool(force or extra_flags or not _same(stamp, listing) or _stale(LIB, _deps()))
    torch = _torch()
    calls_stamp, calls_made_with = os.path.join(BUILD, "calls.txt"), torch and "torch " + torch[1]
    calls_due = torch is not None and bool(force or extra_flags or not _same(calls_stamp, calls_made_with) or
                                           _stale(CALLS, _binding_deps()))
    if not lib_due and not calls_due:
        return LIB
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, torch[0]) if calls_due else None
        results = list(ex.map(lambda s: _compile(s, extra_flags), srcs)) if lib_due else []
    if lib_due:
        if verbose:
            for _, log in results:
                if log:
                    sys.stderr.write(log)
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = ([nvcc()] + ARCH + ["-shared", "-cudart", "static", "-Xlinker", "-soname=libspec_attn.so", "-o", tmp] +
               [o for o, _ in results])
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
        with open(stamp, "w") as f:
            f.write(listing)
    if calls_due:
        try:
            _link_binding(binding.result(), torch[0])
        except Exception:
            if os.path.exists(CALLS):      # (an older one, or another torch's, would be imported in its place)
                os.remove(CALLS)
            raise
        with open(calls_stamp, "w") as f:
            f.write(calls_made_with)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force=True, verbose=v, extra_flags=["-Xptxas", "-v"] if v else []))
