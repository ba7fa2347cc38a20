"""In-tree build of libkda.so (CUDA, sm_103a only) and of the C++ half of its Python binding.

Each ``csrc/*.cu`` translation unit is compiled in parallel with nvcc for
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``linear_attention_06_gb300/libkda.so``; ``csrc/latent_binding.cpp`` is compiled
against the installed torch into ``linear_attention_06_gb300/_latent.so``.  Objects go
to ``_build/``.  No cmake.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "_latent.so")
STAMP = os.path.join(BUILD, "latent_binding.txt")    # what the binding was compiled against
HEADERS = [os.path.join(ROOT, "include", "kda.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _remove(*paths):
    for path in paths:
        if os.path.exists(path):
            os.remove(path)


def _built_for():
    import torch
    return f"torch {torch.__version__} python {sys.version}\n"


def _start_binding(force: bool):
    """Start compiling the C++ binding of the latent-attention entry points against the installed torch, if it is
    stale; returns (its source, the process or None).  An older binding and its stamp go first, and the new ones
    come after success (_finish_binding): a compilation that is cut short leaves nothing that could be loaded."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    src = os.path.join(CSRC, "latent_binding.cpp")
    same = os.path.exists(STAMP) and open(STAMP).read() == _built_for()
    if not force and same and not _stale(BINDING, [src] + HEADERS):
        return src, None
    _remove(STAMP, BINDING)
    inc = cpp_extension.include_paths() + ["/usr/local/cuda/include", sysconfig.get_paths()["include"],
                                           os.path.join(ROOT, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for i in inc for x in ("-isystem", i)] + [src, "-o", os.path.join(BUILD, "latent_binding.so")]
    cmd += [f"-L{p}" for p in cpp_extension.library_paths()]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    return src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish_binding():
    os.replace(os.path.join(BUILD, "latent_binding.so"), BINDING)
    with open(STAMP, "w") as f:
        f.write(_built_for())


def build(force: bool = False, verbose: bool = False, extra_flags=None, tag=None) -> str:
    """Compile (if stale) and return the path of libkda.so.

    With ``tag`` the objects and the library go to ``_build/<tag>/`` instead (a
    separately configured copy, e.g. a diagnostic build with extra ``-D`` flags);
    the package's own ``libkda.so`` is left alone."""
    obj_dir = os.path.join(BUILD, tag) if tag else BUILD
    lib = os.path.join(obj_dir, "libkda.so") if tag else LIB
    os.makedirs(obj_dir, exist_ok=True)
    deps_common = HEADERS + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    flags = CFLAGS + list(extra_flags or [])
    procs, objs = [], []
    for src in sources():
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps_common):
            cmd = [NVCC] + ARCH + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    if not tag:
        src, p = _start_binding(force)
        if p is not None:
            procs.append((src, p))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
            continue
        if src.endswith(".cpp"):
            _finish_binding()
        if verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(f"{s}\n{o}" for s, o in failed))
    if force or _stale(lib, objs):
        cmd = [NVCC] + ARCH + ["-shared", "-o", lib] + objs
        subprocess.run(cmd, check=True)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
