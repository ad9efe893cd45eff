"""Build the CUDA library libssd_gb300.so in-tree (nvcc, sm_103a only).

Each translation unit under csrc/ is compiled in parallel, then linked with a
static CUDA runtime into one shared library next to this file.  The library
has a plain C ABI (include/ssd.h) and no link-time dependency on libcuda (the
driver entry point for tensor-map encoding is looked up at run time).

csrc/binding.cpp (the layer operators on torch tensors) is compiled beside it
into the Python module _layer_binding.so, against the installed torch and the
library.

Run as a script (``python mamba_ssd_forward_chunked_gb300/build_ext.py``) or
load it by path: importing the package itself needs the library it builds.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libssd_gb300.so")
BINDING = os.path.join(HERE, "_layer_binding.so")
BUILD = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _binding_compile(src: str, obj: str):
    """The host compiler's command for the binding (torch is only located, not imported)."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wno-deprecated-declarations",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(cuda, "include"), "-c", src, "-o", obj]


def _binding_link(obj: str, out: str):
    lib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-o", out, obj, "-L", HERE, "-l:" + os.path.basename(OUT),
            "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _binding_made_for(cmds) -> str:
    """What the binding depends on beside its sources: the commands, this Python
    and the installed torch, whose files may be older than what was built."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    with open(os.path.join(torch, "version.py")) as f:
        return "\n".join([sys.version, f.read(), *(" ".join(cmd) for cmd in cmds)])


def _read(path: str):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(what + " failed")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "ssd.h"))
    flags = NVCC_FLAGS + list(extra_flags or [])
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([nvcc, *ARCH, *flags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj])
    binding_src = os.path.join(CSRC, "binding.cpp")
    binding_obj = os.path.join(BUILD, "binding.o")
    binding = [_binding_compile(binding_src, binding_obj), _binding_link(binding_obj, BINDING + ".tmp")]
    made_for, note = _binding_made_for(binding), os.path.join(BUILD, "binding.txt")
    other = _read(note) != made_for
    if force or other or _stale(binding_obj, [binding_src, os.path.join(INCLUDE, "ssd.h")]):
        jobs.append(binding[0])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compilation failed: " + " ".join(cmd))
    if force or jobs or _stale(OUT, objs):
        _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", OUT + ".tmp", *objs], "link")
        os.replace(OUT + ".tmp", OUT)
    if force or other or _stale(BINDING, [binding_obj, OUT]):
        _run(binding[1], "link of the binding")
        os.replace(BINDING + ".tmp", BINDING)
        with open(note, "w") as f:
            f.write(made_for)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
