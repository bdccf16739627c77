"""Build libtreeverify.so in-tree for sm_103a with nvcc.

Each translation unit under csrc/ is compiled in parallel, then linked into
``speculative_decoding_tree_build_gb300/libtreeverify.so``. csrc/binding.cpp is
compiled with the host compiler against torch's headers and linked to it as
the extension module ``_treeverify_torch.so``. The library needs neither torch
nor Python's headers and is there whether or not the extension module compiles;
``--library-only`` leaves that out. Stamps of the sources and flags (and of
torch's version) skip what has not changed.

    python -m speculative_decoding_tree_build_gb300.build [--force] [--verbose-ptxas] [--library-only]

or, where torch is not installed, ``python speculative_decoding_tree_build_gb300/build.py --library-only``.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtreeverify.so")
EXT = os.path.join(PKG, "_treeverify_torch.so")
HEADER = os.path.join(ROOT, "include", "treeverify.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _hash(files, words):
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(words).encode())
    return h.hexdigest()


def _stamp(extra):
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    return _hash(_sources() + headers + [HEADER], ARCH + NVCC_FLAGS + extra)


def _stamp_binding():
    import torch

    return _hash([os.path.join(CSRC, "binding.cpp"), HEADER], [torch.__version__, sys.version])


def _built(target, name, stamp):
    """Whether `target` is there, made from what `stamp` stands for."""
    path = os.path.join(BUILD, name)
    if not (os.path.exists(target) and os.path.exists(path)):
        return False
    with open(path) as fh:
        return fh.read() == stamp


def _note(name, stamp):
    with open(os.path.join(BUILD, name), "w") as fh:
        fh.write(stamp)


def _torch_dirs():
    import torch

    root = os.path.dirname(torch.__file__)
    return os.path.join(root, "include"), os.path.join(root, "lib")


def _compile_binding(nvcc):
    """csrc/binding.cpp -> object file."""
    import torch

    include, _ = _torch_dirs()
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DTV_TORCH_VERSION="{torch.__version__}"',
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding does not compile:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_binding(obj):
    _, lib = _torch_dirs()
    tmp = EXT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-ltreeverify",
           "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding does not link:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, EXT)


def build(force=False, verbose_ptxas=False, quiet=True, bindings=True):
    """Compile and link the library (and the extension module over it, unless
    ``bindings`` is false); returns the library's path."""
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    os.makedirs(BUILD, exist_ok=True)
    stamp = _stamp(extra)
    library = force or not _built(LIB, "stamp", stamp)
    if not library and not bindings:
        return LIB
    stamp_binding = _stamp_binding() if bindings else ""
    extension = bindings and (force or not _built(EXT, "stamp_binding", stamp_binding))
    if not library and not extension:
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if (verbose_ptxas or not quiet) and (res.stdout or res.stderr):
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding, nvcc) if extension else None
        if library:
            objs = list(ex.map(compile_one, _sources()))
            tmp = LIB + ".tmp"
            cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
            os.replace(tmp, LIB)
            _note("stamp", stamp)
        if extension:
            _link_binding(binding.result())
            _note("stamp_binding", stamp_binding)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--library-only", action="store_true", help="without the extension module for torch")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas, quiet=False, bindings=not a.library_only))
