"""Builds libmamba2scan.so (the HIP kernels plus the C ABI) for gfx950, in-tree.

    python -m bwd_mamba2_scan_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
SOURCES = ("mamba2_scan.hip", "conv.hip", "grad_clip.hip", "ssm.hip", "ssm_bwd.hip", "delta.hip", "delta_bwd.hip",
           "norm.hip")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmamba2scan.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # Keep the compiler from emitting packed fp32 (v_pk_*_f32) instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature.
    noise = "'-packed-fp32-ops' is not a recognized feature"
    out = "\n".join(ln for ln in proc.stdout.splitlines() if noise not in ln)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed ({proc.returncode}):\n{out}")
    if out.strip():  # warnings
        print(out, file=sys.stderr, flush=True)


def build(verbose: bool = False) -> str:
    """Compile the library; returns its path.  Raises on compiler failure."""
    with tempfile.TemporaryDirectory(prefix="mamba2scan_build_") as tmp:
        objects = [os.path.join(tmp, src + ".o") for src in SOURCES]
        jobs = [[hipcc(), *HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
                for src, obj in zip(SOURCES, objects)]
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as pool:
            for done in [pool.submit(_run, cmd, verbose) for cmd in jobs]:
                done.result()
        out = f"{LIB_PATH}.tmp{os.getpid()}"
        try:
            _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objects, "-o", out], verbose)
            os.replace(out, LIB_PATH)
        finally:
            if os.path.exists(out):
                os.unlink(out)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
