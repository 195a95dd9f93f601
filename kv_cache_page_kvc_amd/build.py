"""Build libkvc.so for gfx950 with hipcc (in-tree, next to this file).

    python -m kv_cache_page_kvc_amd.build
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libkvc.so")
SOURCES = [os.path.join(HERE, "csrc", f)
           for f in ("kvc_host.cpp", "kvc_kernels.hip", "kvc_cache_rows.hip", "kvc_attend.hip")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # binary32 results must be exactly the defined roundings: no contraction
    # into FMA, correctly rounded divide/sqrt (the HIP default, made explicit)
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed-FP32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def build(verbose: bool = False) -> str:
    """Compile the sources side by side, then link them."""
    with tempfile.TemporaryDirectory() as work:
        def run(cmd):
            if verbose:
                print(" ".join(cmd), flush=True)
            return subprocess.run(cmd, capture_output=True, text=True)

        objects = [os.path.join(work, os.path.basename(f) + ".o") for f in SOURCES]
        compile_flags = [f for f in FLAGS if f != "-shared"] + ["-I", os.path.join(ROOT, "include"),
                                                                "-I", os.path.join(HERE, "csrc"), "-c"]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            done = list(pool.map(lambda fo: run([HIPCC, *compile_flags, "-o", fo[1], fo[0]]), zip(SOURCES, objects)))
        tmp = LIB + ".tmp"
        if all(r.returncode == 0 for r in done):
            done.append(run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objects]))
        if any(r.returncode != 0 for r in done):
            sys.stderr.write("".join(r.stdout + r.stderr for r in done))
            raise RuntimeError("hipcc failed building libkvc.so")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
