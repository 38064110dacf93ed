"""Build step for the HIP libraries (liblora.so and libstep.so, gfx950) next to this file.

    python -m tenant_lora_serving_amd.build

Compiles every source under csrc/ with hipcc into objects under _build/ (in
parallel) and links them into tenant_lora_serving_amd/liblora.so (the routed
delta) and libstep.so (the serving-step operators).  Packed FP32
instructions are turned off for the device code (-packed-fp32-ops): the
compiler otherwise forms them from plain float code.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "liblora.so")
STEP_LIB = os.path.join(HERE, "libstep.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["meta.hip", "delta.hip", "fused_dense.hip", "fused_moe.hip", "fused_moe_w2.hip", "noalloc.hip",
           "abi.cpp", "plan.cpp"]
STEP_SOURCES = ["step_norm.hip", "step_linear.hip", "step_linear_tiled.hip", "step_score.hip", "append.hip",
                "attend_few.hip", "attend_many.hip", "step_abi.cpp", "attend_abi.cpp", "step_plan.cpp"]
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", os.path.join(ROOT, "include"),
               "-D__HIP_PLATFORM_AMD__", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(ln for ln in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in ln and ln.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if out:
        print(out, file=sys.stderr)
    return obj


def _link(objs: list, lib: str):
    tmp = lib + ".tmp"
    subprocess.run([HIPCC, "-shared", f"--offload-arch={ARCH}", *objs, "-o", tmp], check=True)
    os.replace(tmp, lib)


def build(verbose: bool = True) -> str:
    """Compile every source (always) and link liblora.so and libstep.so."""
    os.makedirs(BUILD, exist_ok=True)
    every = SOURCES + STEP_SOURCES
    with ThreadPoolExecutor(max_workers=len(every)) as ex:
        objs = dict(zip(every, ex.map(_compile, every)))
    for lib, sources in ((LIB, SOURCES), (STEP_LIB, STEP_SOURCES)):
        _link([objs[src] for src in sources], lib)
        if verbose:
            print(f"built {lib}")
    return LIB


if __name__ == "__main__":
    build()
