"""Build the gfx950 HIP library libgdntree.so in-tree with hipcc.

    python tree_masked_gated_amd/build.py

Every HIP source is compiled for gfx950 only, with packed-fp32 instruction
selection disabled (the kernels are written for plain fp32 VALU and MFMA).
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgdntree.so")
OBJDIR = os.path.join(ROOT, "_build")

SOURCES = ["abi.hip", "verify_generic.hip", "verify_tiled.hip", "verify_large.hip", "commit.hip", "build.hip",
           "accept.hip", "attn_abi.hip", "attn_rope.hip", "attn_pages.hip",
           "attn_verify_bf16_64.hip", "attn_verify_bf16_128.hip", "attn_verify_bf16_256.hip",
           "attn_verify_f32_64.hip", "attn_verify_f32_128.hip", "attn_verify_f32_256.hip",
           "rule_abi.hip", "rule_step.hip", "rule_bf16_64.hip", "rule_bf16_128.hip", "rule_bf16_256.hip",
           "rule_f32_64.hip", "rule_f32_128.hip", "rule_f32_256.hip", "score.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", f"-I{INCLUDE}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function"]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in p.stderr.splitlines() if noise not in l)
    if p.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(jobs: int = 8) -> str:
    """Compile every source and link libgdntree.so; returns its path."""
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
