"""Compile the CUDA library in-tree: csrc/*.cu -> libb2g_sgemm.so (sm_103a only).

Each translation unit is compiled in parallel with nvcc, then linked into one
shared library with the CUDA runtime linked statically.  `-Xptxas -v` output
(registers, spills, shared memory per kernel) is kept in build/ptxas_<tu>.log,
and the build fails when ptxas reports a register spill in any kernel: the
packed FFMA kernels are capped at 128 registers to keep three CTAs per SM, and
a spill there would otherwise show up only as a quiet loss of speed.

csrc/train_binding.cpp, the native side of the tensor calls in train.py, is
compiled next to them with the host compiler against the installed torch and
linked into _train_binding.so.  The library needs neither: where torch is not
installed it is built alone, and it is linked before a failure of the binding is
reported.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "build")
LIB = os.path.join(PKG, "libb2g_sgemm.so")
BINDING = os.path.join(PKG, "_train_binding.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _newer(path) -> bool:
    """Whether `path` is newer than every source."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _torch_stamp():
    """Which torch is installed (found without importing it); None where there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{version} {spec.origin}"


def _binding_up_to_date() -> bool:
    """The binding is newer than its sources and linked against the torch that is there."""
    stamp = _torch_stamp()
    if stamp is None:
        return True  # nothing to bind to
    try:
        with open(os.path.join(BUILD, "binding_torch.txt")) as f:
            return f.read() == stamp and _newer(BINDING)
    except FileNotFoundError:
        return False


def up_to_date() -> bool:
    return _newer(LIB) and _binding_up_to_date()


_SPILL = re.compile(r"(\d+) bytes spill stores, (\d+) bytes spill loads")
_ENTRY = re.compile(r"Function properties for (\S+)")


def spills(log_text: str):
    """[(function, spill store bytes, spill load bytes)] for every function
    whose ptxas report shows a spill."""
    out, fn = [], None
    for line in log_text.splitlines():
        m = _ENTRY.search(line)
        if m:
            fn = m.group(1)
            continue
        m = _SPILL.search(line)
        if m and (int(m.group(1)) or int(m.group(2))):
            out.append((fn, int(m.group(1)), int(m.group(2))))
    return out


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src[:-3] + ".o")
    log = os.path.join(BUILD, f"ptxas_{src[:-3]}.log")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr[-4000:]}")
    bad = spills(r.stdout + r.stderr)
    if bad:
        os.remove(obj)
        raise RuntimeError(f"ptxas reports register spills in {src}: " +
                           "; ".join(f"{f}: {st} B stored, {ld} B loaded" for f, st, ld in bad))
    return obj


def _torch_paths():
    """(include, library) directories of the installed torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    return ([os.path.join(root, "include"),
             os.path.join(root, "include", "torch", "csrc", "api", "include")],
            os.path.join(root, "lib"))


def _compile_binding() -> str:
    """csrc/train_binding.cpp -> build/train_binding.o."""
    import torch

    cxx = shutil.which("g++") or "g++"
    obj = os.path.join(BUILD, "train_binding.o")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    cmd = [cxx, "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE, "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"]]
    for d in _torch_paths()[0]:
        cmd += ["-isystem", d]
    cmd += ["-c", os.path.join(CSRC, "train_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on train_binding.cpp:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    lib = _torch_paths()[1]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lb2g_sgemm",
           "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, BINDING)
    with open(os.path.join(BUILD, "binding_torch.txt"), "w") as f:
        f.write(_torch_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build the library and the binding if any source is newer, or the binding's torch
    another one; return the library's path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding) if _torch_stamp() else None
        if force or not _newer(LIB):
            objs = list(ex.map(_compile, srcs))
            tmp = LIB + f".tmp{os.getpid()}"
            cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
            os.replace(tmp, LIB)
    if binding:
        _link_binding(binding.result())
    if verbose:
        for s in srcs:
            with open(os.path.join(BUILD, f"ptxas_{s[:-3]}.log")) as f:
                sys.stdout.write(f.read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
