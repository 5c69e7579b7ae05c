"""In-tree build of libattn.so for sm_103a (nvcc, no cmake).

``python -m attention_forward_07_gb300.build`` or ``__graft_entry__.build()``.
The shared library lands next to this file; it is git-ignored.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("attn_fwd.cu", "paged_attn.cu", "paged_tile.cu", "paged_cache.cu", "paged_tree.cu", "rope.cu")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in ("ptx.cuh", "host.h", "roles.cuh", "paged.cuh")] + [os.path.join(ROOT, "include", "attn.h")]
OUT = os.path.join(HERE, "libattn.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(s) <= t for s in SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    if verbose:
        cmd.insert(2, "-Xptxas=-v")
    objects = [tmp + f".{i}.o" for i in range(len(SOURCES))]
    try:
        # the sources side by side, then the link
        jobs = [subprocess.Popen(cmd + ["-c", s, "-o", o], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                for s, o in zip(SOURCES, objects)]
        outs = [j.communicate()[0] for j in jobs]
        failed = any(j.returncode != 0 for j in jobs)
        if not failed:
            r = subprocess.run(cmd + ["-shared", "-o", tmp, *objects], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            outs.append(r.stdout)
            failed = r.returncode != 0
        if failed or verbose:
            sys.stderr.write("".join(outs))
        if failed:
            raise RuntimeError("nvcc failed building libattn.so")
        os.replace(tmp, OUT)
    finally:
        for f in objects:
            if os.path.exists(f):
                os.remove(f)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
