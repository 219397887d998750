"""Build libgdn.so in-tree with nvcc for sm_103a.

Each .cu translation unit is compiled in parallel to an object under
``_build/`` at the repository root, then linked into
``gated_deltanet_linear_16_gb300/libgdn.so`` (CUDA runtime linked statically,
only the symbols of include/gdn.h, include/gdna.h and include/gdnb.h exported).  Rebuilds only when a
source, the public header or the flags changed.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-I" + INCLUDE, "-I" + CSRC,
]
LINK_FLAGS = ARCH + ["-shared", "-cudart", "static"]
SOURCES = ["gdn_abi.cu", "gdn_decode.cu", "gdn_chunk2.cu", "gdn_conv_norm.cu", "gdn_prefill.cu", "gdn_convert.cu",
           "gdn_noalloc.cu", "gdn_norm.cu", "gdn_prefill_tc.cu",
           "gdna_abi.cu", "gdna_pages.cu", "gdna_rope.cu", "gdna_attn.cu",
           "gdna_attn_f16.cu", "gdna_attn_bf16.cu", "gdna_attn_e4m3.cu",
           "gdnb_abi.cu", "gdnb_norm.cu", "gdnb_join.cu", "gdnb_flash_64_f16.cu", "gdnb_flash_64_bf16.cu",
           "gdnb_flash_128_f16.cu", "gdnb_flash_128_bf16.cu", "gdnb_flash_256_f16.cu", "gdnb_flash_256_bf16.cu"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn")
    return exe


def _stamp() -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS + LINK_FLAGS).encode())
    for name in sorted(os.listdir(CSRC)) + ["../../include/gdn.h", "../../include/gdna.h", "../../include/gdnb.h"]:
        path = os.path.normpath(os.path.join(CSRC, name))
        if os.path.isfile(path):
            h.update(name.encode())
            with open(path, "rb") as f:
                h.update(f.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libgdn.so if anything changed; returns its path."""
    stamp_path = LIB + ".stamp"
    stamp = _stamp() + "|" + " ".join(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(stamp_path):
        with open(stamp_path) as f:
            if f.read() == stamp:
                return LIB
    os.makedirs(BUILD, exist_ok=True)
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [exe, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([exe, *LINK_FLAGS, *objs, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_path, "w") as f:
        f.write(stamp)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else ()))
