"""Compiles the gfx950 HIP libraries in-tree with hipcc: libmxfp8.so (the
casts and their consumer, behind include/mxfp8.h), libmxtrain.so (the 16- and
32-bit operators of a training step beside them, behind include/mxtrain.h and
include/mxtrain_tokens.h) and
libmxstream.so (the streaming bandwidth probe behind include/mxstream.h,
measurement only)."""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libmxfp8.so")
SOURCES = [os.path.join(CSRC, "mxfp8.hip")]
STREAM_LIB_PATH = os.path.join(PKG_DIR, "libmxstream.so")
STREAM_SOURCES = [os.path.join(CSRC, "mx_stream.hip")]
TRAIN_LIB_PATH = os.path.join(PKG_DIR, "libmxtrain.so")
TRAIN_SOURCES = [os.path.join(CSRC, "train", name) for name in (
    "mxtrain.hip", "mxtrain_gemm.hip", "mxtrain_ortho.hip", "mxtrain_ortho_bf16.hip", "mxtrain_ortho_f32.hip",
    "mxtrain_sort.hip", "mxtrain_route.hip", "mxtrain_embed.hip", "mxtrain_dropout.hip")]
ARCH = "gfx950"


def kernel_source_hash() -> str:
    """Short hash of the kernel sources of libmxfp8.so and libmxstream.so
    (the .hip/.hpp/.h files directly under csrc/): ties a recorded profile
    to the code it measured."""
    h = hashlib.sha256()
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".hip", ".hpp", ".h")):
            continue
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    return h.hexdigest()[:16]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libmxfp8.so)")


def compile_flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}",
        "-O3",
        "-std=c++17",
        "-fPIC",
        # keep fp32 math scalar: no packed-fp32 instructions are generated
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall",
        "-I", INCLUDE,
        "-I", CSRC,
    ]


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so
    noise = "'-packed-fp32-ops' is not a recognized feature"
    text = "\n".join(l for l in res.stdout.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{text}")
    if verbose and text.strip():
        print(text, flush=True)


def build(out: str = LIB_PATH, extra_flags: list[str] | None = None, verbose: bool = False,
          sources: list[str] | None = None) -> str:
    """Compiles `sources` into the shared library `out`; several sources are
    compiled side by side and linked."""
    tmp = out + ".tmp"
    sources = sources or SOURCES
    flags = [*compile_flags(), *(extra_flags or [])]
    if len(sources) == 1:
        _run([hipcc(), *flags, "-shared", "-o", tmp, *sources], verbose)
    else:
        with tempfile.TemporaryDirectory() as d:
            objects = [os.path.join(d, os.path.basename(s) + ".o") for s in sources]
            with ThreadPoolExecutor(max_workers=min(len(sources), 8)) as pool:
                for _ in pool.map(lambda so: _run([hipcc(), *flags, "-c", "-o", so[1], so[0]], verbose),
                                  zip(sources, objects)):
                    pass
            _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-o", tmp, *objects], verbose)
    os.replace(tmp, out)
    return out


def build_all(verbose: bool = False) -> None:
    build(verbose=verbose)
    build(TRAIN_LIB_PATH, verbose=verbose, sources=TRAIN_SOURCES)
    build(STREAM_LIB_PATH, verbose=verbose, sources=STREAM_SOURCES)


if __name__ == "__main__":
    build_all(verbose=True)
