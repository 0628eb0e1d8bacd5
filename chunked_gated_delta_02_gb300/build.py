"""Build libkda.so (sm_103a) in-tree with nvcc, and the native binding of the serving operators.

Every .cu file under csrc/ is compiled to an object in parallel, then linked
into chunked_gated_delta_02_gb300/libkda.so; binding.cpp is compiled beside them
with the host compiler against the installed torch, and linked with libkda.so
into the extension module _serving; where there is no torch, libkda.so is all
that is built. Only one -gencode target is
built: compute_103a / sm_103a (the arch-specific variant is needed for the
tcgen05 and TMA instructions).
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "_serving.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put /usr/local/cuda/bin on PATH)")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir():
    """The installed torch's folder, or None."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else os.path.dirname(spec.origin)


def _binding_compile(obj):
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
            "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj, "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]


def _binding_link(obj, target):
    libs = os.path.join(_torch_dir(), "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-o", target, obj, "-L" + PKG, "-l:libkda.so", "-L" + libs,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _note_torch(path):
    """Writes which torch and Python the binding is built against, if `path` does not say so yet."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        text = "\n".join((_torch_dir(), sys.version, f.read()))
    if os.path.exists(path):
        with open(path) as f:
            if f.read() == text:
                return
    with open(path, "w") as f:
        f.write(text)


def _link(target, deps, command, force):
    if force or _stale(target, deps):
        tmp = target + f".tmp{os.getpid()}"
        r = subprocess.run(command(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link libkda.so, then the binding where torch is installed; returns the library's path.

    Raises on a compiler error; one in the binding leaves the library in place.
    """
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(os.path.dirname(PKG), "include", "*.h"))
    objs, procs = [], []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc()] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + \
                ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    binding_src = os.path.join(CSRC, "binding.cpp")
    binding_obj = os.path.join(BUILD, "binding.cpp.o")
    binding_torch = os.path.join(BUILD, "binding.torch")
    with_binding = _torch_dir() is not None
    if with_binding:
        _note_torch(binding_torch)
    if with_binding and (force or _stale(binding_obj, [binding_src, binding_torch] + headers)):
        cmd = _binding_compile(binding_obj)
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((binding_src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = {}
    for src, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed[src] = f"--- {src}\n{text}"
        elif verbose or ptxas_verbose:
            sys.stderr.write(text)
    binding_failed = failed.pop(binding_src, None)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed.values()))
    _link(LIB, objs, lambda tmp: [nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=libkda.so", "-o", tmp] + objs + ["-lcudart"],
          force)
    if binding_failed:
        raise RuntimeError("the binding failed to compile:\n" + binding_failed)
    if with_binding:
        _link(BINDING, [binding_obj, LIB], lambda tmp: _binding_link(binding_obj, tmp), force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
