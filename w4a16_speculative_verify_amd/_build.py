"""Build libw4v.so for gfx950 with hipcc (in-tree, next to this file)."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4v.so")

SOURCES = ["w4a16_skinny.hip", "w4a16_mfma.hip", "w4a16_chain.hip",
           "w8a16_lmhead.hip", "greedy_verify.hip", "ngram_draft.hip", "gdn_commit.hip",
           "gdn_forward.hip", "rope_append.hip", "paged_attention.hip", "read_probe.hip", "lib_gemm.cpp",
           "api.cpp"]
# the vendor GEMM library behind the fp16 linear (f16_gemm) only
LIBS = ["-L/opt/rocm/lib", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"]

# gfx950 only.  Packed-fp32 instructions are switched off for every HIP
# translation unit (the host pass reports the feature as unknown; harmless).
# MFMA accumulators stay in ordinary VGPRs (no copies out of AGPRs before the
# per-group scale is applied).
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-function",
]


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libw4v)")


# per-source flags: the skinny W4A16 kernel takes its first 14 argument dwords
# preloaded into SGPRs (the scalars its first group step needs)
SOURCE_FLAGS = {"w4a16_skinny.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=14"]}


def _compile(src: str, hipcc: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc, *HIP_FLAGS, *SOURCE_FLAGS.get(src, []), "-x", "hip", "-I", INCLUDE, "-I", CSRC,
           "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        msg = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                        if "packed-fp32-ops" not in l)
        if msg.strip():
            print(msg)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{' '.join(cmd)}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link libw4v.so; returns the library path."""
    hipcc = _hipcc()
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as pool:
        objs = list(pool.map(lambda s: _compile(s, hipcc, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, *LIBS, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
