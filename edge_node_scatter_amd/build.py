"""Compile libzs.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

The library is built in-tree next to this file.  Compiler flags that matter
for results:

* ``-ffp-contract=off``: fp32 multiplies and adds stay separately rounded, as
  in the materialised-message reference; the fp64 channel sums use explicit
  ``fma`` calls, which this flag does not affect.
* ``-fno-gpu-flush-denormals-to-zero``: fp32 subnormals are kept (IEEE).
* ``-Xclang -target-feature -Xclang -packed-fp32-ops``: no packed fp32 VALU
  instructions are generated.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libzs.so")
SOURCES = ["zs_api.hip", "zs_csr.hip", "zs_fwd.hip", "zs_bwd.hip", "zs_norm.hip",
           "zs_block_api.hip", "zs_gmm.hip", "zs_wgrad.hip", "zs_join.hip", "zs_adamw.hip",
           "zs_layers_api.hip", "zs_embed.hip", "zs_lnorm.hip", "zs_route.hip", "zs_combine.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-fast-math", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


JOBS = 8   # sources compiled at a time


def _run(cmd: list[str], verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)


def build(verbose: bool = False) -> str:
    """Compile every source into libzs.so (always recompiles)."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory(prefix="zs_build_") as objs:
        cmds, names = [], []
        for s in SOURCES:
            names.append(os.path.join(objs, s.replace(".hip", ".o")))
            cmds.append([HIPCC, *[f for f in FLAGS if f != "-shared"], "-c", os.path.join(CSRC, s),
                         "-o", names[-1]])
        with ThreadPoolExecutor(JOBS) as pool:
            list(pool.map(lambda c: _run(c, verbose), cmds))
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *names, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


def device_asm(out_dir: str) -> list[str]:
    """Write the gfx950 assembly of every kernel source (for instruction checks)."""
    os.makedirs(out_dir, exist_ok=True)
    paths = [os.path.join(out_dir, s.replace(".hip", f"-{ARCH}.s")) for s in SOURCES]
    flags = [f for f in FLAGS if f not in ("-shared", "-fPIC")]
    cmds = [[HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(CSRC, s), "-o", out]
            for s, out in zip(SOURCES, paths)]
    with ThreadPoolExecutor(JOBS) as pool:
        list(pool.map(_run, cmds))
    return paths


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
