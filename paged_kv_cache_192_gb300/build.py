"""Build the sm_103a shared library libpa_gb300.so in-tree.

Each translation unit under csrc/ is compiled by nvcc in parallel, then the
objects are linked into ``paged_kv_cache_192_gb300/libpa_gb300.so`` (static
CUDA runtime, no torch dependency).  Where torch is installed,
``binding/bounded_calls.cpp`` (the torch-facing binding of the calls whose time
on the host counts) then becomes the extension module ``_bounded_calls.so``,
linked to the library and to that torch; it also needs g++ and the Python
headers.  The library needs none of them and is linked first.  Objects are
cached in ``_build/`` keyed by a hash of the sources and flags, so an unchanged
tree rebuilds in no time.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa_gb300.so")
BINDING_SRC = os.path.join(PKG, "binding", "bounded_calls.cpp")
BINDING = os.path.join(PKG, "_bounded_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _digest(paths, extra) -> str:
    h = hashlib.sha1()
    for p in sorted(paths):
        with open(p, "rb") as f:
            h.update(p.encode() + b"\0" + f.read())
    h.update(" ".join(extra).encode())
    return h.hexdigest()[:16]


def _torch_flags():
    """(compile flags, link flags, version) of an extension module of the
    running Python against the installed torch (found without importing it);
    None without one."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    root = os.path.dirname(spec.origin)
    with open(os.path.join(root, "version.py")) as f:
        version = f.read()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    comp = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + [x for i in inc for x in ("-I", i)]
    lib = os.path.join(root, "lib")
    link = ["-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10",
            f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    return comp, link, version


def _compile_binding(src: str, obj: str, flags) -> str:
    if os.path.exists(obj):
        return obj
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found")
    tmp = obj + ".tmp.o"
    r = subprocess.run([cxx] + flags + ["-c", src, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, obj)
    return obj


def _compile(src: str, obj: str, headers) -> str:
    if os.path.exists(obj):
        return obj
    tmp = obj + ".tmp.o"
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, obj)
    return obj


def _link(out: str, cmd, objs, libs, stamp_name: str) -> bool:
    """Links out unless it is there already; whether it was linked."""
    key = _digest(objs, cmd + libs)
    stamp = os.path.join(BUILD, stamp_name)
    if os.path.exists(out) and os.path.exists(stamp) and open(stamp).read() == key:
        return False
    tmp = out + ".tmp"
    r = subprocess.run(cmd + ["-o", tmp] + objs + libs, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(out)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    with open(stamp, "w") as f:
        f.write(key)
    return True


def build(verbose: bool = False) -> str:
    """Compile and link the library, and the binding where torch is installed;
    returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                     glob.glob(os.path.join(INCLUDE, "*.h")))
    hdr_digest = _digest(headers, NVCC_FLAGS)
    objs, binding_obj = [], None
    torch_flags = _torch_flags()
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        futs = []
        for src in sources:
            key = _digest([src], [hdr_digest])
            obj = os.path.join(BUILD, f"{os.path.basename(src)}.{key}.o")
            objs.append(obj)
            futs.append(ex.submit(_compile, src, obj, headers))
        if torch_flags:
            comp, link, torch_version = torch_flags
            key = _digest([BINDING_SRC] + headers, comp + [torch_version])
            binding_obj = os.path.join(BUILD, f"bounded_calls.cpp.{key}.o")
            binding_done = ex.submit(_compile_binding, BINDING_SRC, binding_obj, comp)
        for f in futs:
            f.result()
    # objects of earlier sources or flags are not reused: drop them
    keep = {os.path.basename(o) for o in objs + ([binding_obj] if binding_obj else [])}
    for old in glob.glob(os.path.join(BUILD, "*.o")):
        if os.path.basename(old) not in keep:
            os.remove(old)
    if _link(LIB, [nvcc()] + ARCH + ["-shared"], objs, ["-lpthread"], "lib.stamp"):
        # a binding of an earlier library does not outlive it
        if os.path.exists(BINDING):
            os.remove(BINDING)
    if binding_obj:
        binding_done.result()
        # (the library is found beside the module; its name is what the loader sees)
        _link(BINDING, [shutil.which("g++") or "c++", "-shared"], [binding_obj],
              ["-L", PKG, "-l:" + os.path.basename(LIB)] + link, "binding.stamp")
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
