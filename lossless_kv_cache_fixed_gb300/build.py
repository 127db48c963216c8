"""Build libskv.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs)."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libskv.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["skv_code.cu", "skv_bits.cu", "skv_scale.cu", "skv_adapt.cu", "skv_api.cu",
           "skv_cache_pages.cu", "skv_cache_append.cu", "skv_cache_attend.cu", "skv_cache_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "skv.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def source_digest() -> str:
    """Hash of the coder's kernel sources, to tie its measurements to the code they
    describe (the paged cache's sources, skv_cache*, are not part of the coder)."""
    import hashlib
    h = hashlib.sha256()
    for f in sorted(f for f in os.listdir(CSRC) if not f.startswith("skv_cache")):
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + b"\0" + fh.read())
    return h.hexdigest()[:16]


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps():
        return LIB
    flags = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE] + ARCH
    if ptxas_v:
        flags += ["-Xptxas", "-v"]
    tag = "%d" % os.getpid()

    def compile_one(src):
        obj = os.path.join(OUT, src.replace(".cu", ".%s.o" % tag))
        cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_v:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s" % src)
        return obj

    tmp = LIB + ".tmp" + tag
    leftovers = [os.path.join(OUT, src.replace(".cu", ".%s.o" % tag)) for src in SOURCES] + [tmp]
    try:
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            objs = list(ex.map(compile_one, SOURCES))
        cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    finally:
        # this build's objects and temporary library go, whether it succeeded or not
        for f in leftovers:
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
