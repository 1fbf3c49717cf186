"""Build libkda_tril.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree.

Usage: python tril_solve_amd/build.py   (run as a script: importing the
package would load the library before it is built)
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libkda_tril.so")
PROBE_LIB = os.path.join(HERE, "libkda_bench_probe.so")
OBJDIR = os.path.join(HERE, "_build")

SOURCES = ["api.cpp", "plan.cpp", "launch_common.cpp", "tril_fused.hip", "tril_split.hip",
           "tril_small.hip", "tril_kkt.hip", "kda_decode.hip", "layer_api.cpp", "kda_map.hip",
           "kda_conv.hip", "kda_prefill.hip", "kda_prefill_f32.hip", "kda_prefill_bf16.hip",
           "kda_prefill_f16.hip", "kda_recurrent.hip", "kda_norm.hip", "grad_api.cpp",
           "kda_delta_grad_f32.hip", "kda_delta_grad_bf16.hip", "kda_delta_grad_f16.hip",
           "kda_conv_grad.hip", "kda_norm_grad.hip", "kda_checkpoint.hip"]
PROBE_SOURCES = ["bench_probe.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# Packed FP32 VALU instructions are disabled for all device code: hipcc would
# otherwise form v_pk_{add,mul,fma}_f32 from scalar float code.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
COMMON = ["-O3", "-std=c++20", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
          "-Wall", "-Wno-unused-function"]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + COMMON + DEVICE_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [HIPCC] + COMMON + ["-x", "hip"] + DEVICE_FLAGS + ["-c", os.path.join(CSRC, src),
                                                                  "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msg}")
    if msg:
        print(msg, file=sys.stderr)
    return obj


def _link(objs, out):
    tmp = out + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    """Compile every source and link the solver library and the benchmark's
    copy probe. Returns the solver library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = SOURCES + PROBE_SOURCES
    with ThreadPoolExecutor(min(8, len(srcs))) as ex:
        objs = dict(zip(srcs, ex.map(_compile, srcs)))
    _link([objs[s] for s in SOURCES], LIB)
    _link([objs[s] for s in PROBE_SOURCES], PROBE_LIB)
    if verbose:
        print(f"built {LIB} and {PROBE_LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
