"""Build libssd.so (the HIP kernels and the C ABI) for gfx950 with hipcc.

    python mamba_ssd_chunked_fwd_amd/build.py

(run by path: importing the package loads the library this script builds)

Sources compile in parallel into objects under _build/ at the repository
root, then link into mamba_ssd_chunked_fwd_amd/libssd.so.  All device code
is built with packed-fp32 instructions disabled.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "libssd")
LIB = os.path.join(PKG, "libssd.so")
ARCH = "gfx950"

SOURCES = ["ssd_api.cpp", "ssd_chunk_cumsum.hip", "ssd_fwd_pass_state.hip",
           "ssd_compute_out.hip", "ssd_decode_step.hip",
           "ssd_causal_conv1d.hip", "ssd_gdn.hip",
           "ssd_state_two_level.hip", "ssd_forward_noalloc.hip",
           "ssd_fused_f32.hip", "ssd_fused_bf16.hip", "ssd_state_pair_f32.hip",
           "ssd_block_api.cpp", "ssd_block_norm.hip", "ssd_linattn.hip",
           "ssd_linattn_step.hip",
           "ssd_selective_api.cpp", "ssd_selective_scan.hip",
           "ssd_selective_scan_bwd.hip", "ssd_selective_step.hip",
           "ssd_short_conv.hip", "ssd_norm_quant.hip"]

HIP_FLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Wno-unused-function"]


def _hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found (ROCm is required to build libssd)")
    return p


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
           os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # The host pass does not know the packed-fp32 feature and says so.
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)
    return obj


def build(verbose: bool = False, jobs: int = 4) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp,
           *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
