"""Build libufp4.so (HIP, gfx950) in-tree with hipcc.

Usage: python -m uniform_grid_fp4_amd.build   (or call build()).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libufp4.so")
SOURCES = ["api.hip", "quantize.hip", "gemm.hip", "stats.hip",
           "block_api.hip", "rmsnorm.hip", "route.hip", "exchange.hip", "gradnorm.hip",
           "ffn_api.hip", "layernorm.hip", "dropout.hip", "gated_small.hip", "gated_bwd.hip",
           "int8_quantize.hip", "int8_gemm.hip"]
# The bench's MFMA issue-rate probe: a separate library, not part of the ABI.
PROBE_LIB = os.path.join(HERE, "libufp4_probe.so")
PROBE_SOURCES = ["probe.hip"]

# -ffp-contract=off: no multiply-add fusion anywhere (the quantizer's two
#   roundings r = RN(g/s), t = RN(y*r) must stay separate).
# -fno-gpu-flush-denormals-to-zero: FP32 subnormals are kept (bf16 inputs and
#   butterfly outputs can be subnormal).
# -packed-fp32-ops disabled: no v_pk_* FP32 instructions are generated.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libufp4.so")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)
    noise = [ln for ln in res.stderr.splitlines()
             if "packed-fp32-ops" not in ln and ln.strip()]
    if noise and verbose:
        print("\n".join(noise), file=sys.stderr)


def _compile(sources, out, verbose):
    """Each source to an object (a few at a time), then one shared library."""
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, s + ".o") for s in sources]
        base = [hipcc(), *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC]
        with ThreadPoolExecutor(max_workers=min(8, len(sources))) as pool:
            list(pool.map(lambda so: _run([*base, "-c", os.path.join(CSRC, so[0]), "-o", so[1]],
                                          verbose), zip(sources, objs)))
        _run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", out + ".tmp"],
             verbose)
    os.replace(out + ".tmp", out)


def build(verbose: bool = False) -> str:
    """Compile every HIP source: libufp4.so and the probe library."""
    _compile(SOURCES, LIB, verbose)
    _compile(PROBE_SOURCES, PROBE_LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
