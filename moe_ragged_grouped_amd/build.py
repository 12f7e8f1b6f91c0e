"""Compile the gfx950 HIP libraries in-tree with hipcc.

    python -m moe_ragged_grouped_amd.build

produces moe_ragged_grouped_amd/libmoe_ragged_grouped_amd.so from csrc/, and
libmoe_ragged_grouped_amd_trace.so, the forward products' source built with
GG_TILE_TRACE (the per-tile timeline of include/grouped_gemm_trace.h; a
diagnostic the product library does not contain).
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
LIB = os.path.join(HERE, "libmoe_ragged_grouped_amd.so")
TRACE_LIB = os.path.join(HERE, "libmoe_ragged_grouped_amd_trace.so")
# the forward products; the tracing build is made of these alone
SOURCES = [os.path.join(CSRC, "grouped_gemm.hip")]
# the gradients and the 4-bit operators
OPERATOR_SOURCES = [os.path.join(CSRC, f) for f in
                    ("grouped_dgrad.hip", "grouped_wgrad.hip", "grouped_mx4.hip")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # hipcc -O3 forms packed fp32 ops from plain float code; keep it from doing so
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (r.stdout + r.stderr).splitlines() if noise not in ln]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


def build(verbose: bool = False, extra=(), out: str = LIB, sources=None) -> str:
    """Compile every source (side by side) and link them into one library."""
    sources = SOURCES + OPERATOR_SOURCES if sources is None else sources
    flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in sources]
        with ThreadPoolExecutor(max_workers=len(sources)) as ex:
            list(ex.map(lambda so: _run([HIPCC, *flags, *extra, "-c", "-o", so[1], so[0]], verbose),
                        zip(sources, objs)))
        tmp = out + ".tmp%d" % os.getpid()
        _run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, out)
    return out


def build_trace(verbose: bool = False) -> str:
    return build(verbose, extra=("-DGG_TILE_TRACE",), out=TRACE_LIB, sources=SOURCES)


if __name__ == "__main__":
    print(build(verbose=True, extra=sys.argv[1:]))
    print(build_trace(verbose=True))
