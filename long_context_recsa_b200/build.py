"""Build librecsa.so in-tree for sm_100a with nvcc.

Usage: python -m long_context_recsa_b200.build   (or build() from Python)
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "librecsa.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["recsa_api.cu", "tree_kernels.cu", "select_attend.cu", "prefill_tc.cu", "noalloc.cu",
           "gated.cu", "offload.cu", "kv4_api.cu", "kv4_rows.cu", "kv4_attend.cu",
           "kv4_chunk.cu", "kv4_evict.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps) -> bool:
    if deps is None or not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _compiled_from(depfile: str):
    """The files that a make-style dependency file lists; None without one."""
    if not os.path.exists(depfile):
        return None
    with open(depfile) as f:
        names = f.read().replace("\\\n", " ").split(":", 1)[-1].split()
    return names if all(os.path.exists(n) for n in names) else None


OUT_BOUNDS = os.path.join(HERE, "librecsa_bounds.so")


def build(force: bool = False, verbose: bool = False, debug_bounds: bool = False) -> str:
    """Compile the library (librecsa.so), or with debug_bounds the bounds-checked
    variant (librecsa_bounds.so: every gather row and selection rank is range-checked
    on the device and a failure is recorded in the status word)."""
    out = OUT_BOUNDS if debug_bounds else OUT
    deps = [os.path.join(CSRC, s) for s in SOURCES]
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(HERE, "..", "include", "recsa.h"))
    flags = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
             "-Xcompiler", "-fvisibility=hidden"]
    if debug_bounds:
        flags.append("-DRECSA_DEBUG_BOUNDS")
    # one object per source, compiled side by side; an object newer than every file it
    # was compiled from (listed in its .d file), and made with the same flags, is kept
    objdir = os.path.join(BUILD, "bounds" if debug_bounds else "release")
    made_with, now = os.path.join(objdir, "flags.txt"), "\n".join([*flags, *SOURCES])
    if not os.path.exists(made_with) or open(made_with).read() != now:
        force = True
    if not force and not _stale(out, deps):
        return out
    os.makedirs(objdir, exist_ok=True)
    if force and os.path.exists(made_with):
        os.remove(made_with)             # until all objects are made anew
    if verbose:
        flags.append("-Xptxas=-v")

    def compile_one(src: str) -> str:
        path = os.path.join(CSRC, src)
        obj = os.path.join(objdir, src + ".o")
        if force or _stale(obj, _compiled_from(obj + ".d")):
            cmd = [nvcc_path(), *flags, "-MD", "-MF", obj + ".d", "-c", "-o", obj + ".tmp", path]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            subprocess.run(cmd, check=True)
            os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, os.cpu_count() or 1)) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    subprocess.run([nvcc_path(), *ARCH, "-shared", "-o", out + ".tmp", *objs], check=True)
    os.replace(out + ".tmp", out)
    with open(made_with, "w") as f:
        f.write(now)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug_bounds="--bounds" in sys.argv))
