"""In-tree build of the CUDA library (``libspecv.so``) for sm_103a.

Translation units (``UNITS``) compiled by nvcc side by side and linked with
the CUDA runtime statically; the result sits next to this file, where the
binding loads it.  Rebuilt when any source or the public header is newer.
"""
import concurrent.futures
import glob
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libspecv.so")
SOURCES = sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")) + glob.glob(os.path.join(PKG, "csrc", "*.cuh")))
UNITS = ("library.cu", "prefix.cu", "serving.cu")
HEADER = os.path.join(ROOT, "include", "specv.h")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecv.so")


def needs_build():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in SOURCES + [HEADER])


def build(force=False, verbose=False):
    """Compile libspecv.so if missing or stale; return its path."""
    if not force and not needs_build():
        return LIB
    flags = [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    tmp = LIB + ".tmp"

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
        if verbose:
            print(res.stdout + res.stderr)

    nvcc = nvcc_path()
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, u + ".o") for u in UNITS]
        with concurrent.futures.ThreadPoolExecutor() as pool:
            list(pool.map(lambda u, o: run([nvcc, *flags, "-c", "-o", o, os.path.join(PKG, "csrc", u)]), UNITS, objects))
        run([nvcc, ARCH, "-shared", "-o", tmp, *objects])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
