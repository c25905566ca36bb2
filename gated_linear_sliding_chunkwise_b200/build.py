"""Build liblizard.so in-tree with nvcc for sm_100a.

    python -m gated_linear_sliding_chunkwise_b200.build [--force] [-v]

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (skipped when
newer than its sources), then linked into ``liblizard.so`` next to this file.
That takes nvcc alone.  ``csrc/paged_binding.cpp`` then becomes the extension
module ``_paged_call.so``, which takes a CUDA build of torch and g++; without
them it is left out, and importing ``.paged`` says so.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "liblizard.so")
BINDING = os.path.join(HERE, "_paged_call.so")   # Python entry of the paged cache

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblizard.so")


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hdrs.append(os.path.join(INCLUDE, "lizard.h"))
    return hdrs


def _stale(target, sources):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cus = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    deps = _deps()
    cc = nvcc()
    jobs = []
    objs = []
    for f in cus:
        src = os.path.join(CSRC, f)
        obj = os.path.join(BUILD, f[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps):
            cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if force or jobs or _stale(LIB, objs):
        cmd = [cc, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    build_binding(force)
    return LIB


def _torch_version():
    """What the extension module is compiled against, without importing it; None without torch."""
    try:
        return f"torch {importlib.metadata.version('torch')}, python {sys.version_info[0]}.{sys.version_info[1]}\n"
    except importlib.metadata.PackageNotFoundError:
        return None


def _without_binding(why: str):
    sys.stderr.write(f"_paged_call.so, the paged cache's Python entry, is left out: {why}\n")


def build_binding(force: bool = False):
    """The extension module of the paged cache: torch's headers, linked to
    liblizard.so beside it.  Compiled again for another torch or Python: the
    one that is there would not fit.  Returns its path, or None where it
    cannot be compiled."""
    src = os.path.join(CSRC, "paged_binding.cpp")
    stamp = os.path.join(BUILD, "paged_call.against")
    against, before = _torch_version(), None
    if os.path.exists(stamp):
        with open(stamp) as f:
            before = f.read()
    if not force and against == before and not _stale(BINDING, [src, os.path.join(INCLUDE, "lizard.h")]):
        return BINDING
    if os.path.exists(BINDING):              # not to be found by an import if it cannot be made anew
        os.remove(BINDING)
    gxx = shutil.which("g++")
    if against is None or gxx is None:
        return _without_binding("torch is not installed" if against is None else "there is no g++")
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    if torch.version.cuda is None:
        return _without_binding("torch is a build without CUDA")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [*ext.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in include), src, "-o", BINDING, f"-L{HERE}", "-llizard", f"-L{libs}", "-ltorch_python",
           "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError("building the binding failed:\n" + r.stdout + r.stderr)
    with open(stamp, "w") as f:
        f.write(against)
    return BINDING


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
