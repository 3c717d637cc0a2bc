"""Build libidxtopk.so for gfx950 with hipcc (in-tree, no JIT cache)."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = ["csrc/idx_api.hip", "csrc/idx_prefill.hip", "csrc/idx_decode.hip", "csrc/idx_rows.hip", "csrc/idx_scan.hip"]
# sources whose masked places may hold NaN: compiled without -fno-honor-nans
NAN_SOURCES = ["csrc/idx_latent.hip", "csrc/idx_expanded.hip", "csrc/idx_norm.hip"]
LIB = os.path.join(HERE, "libidxtopk.so")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
    "-ffp-contract=off",
    # packed FP32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
# inputs are NaN-free by contract: lets max(x, 0) skip a canonicalising op
NO_NANS = "-fno-honor-nans"


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out:
        print(out, flush=True)


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as objs:
        jobs, made = [], []
        for s in SOURCES + NAN_SOURCES:
            obj = os.path.join(objs, os.path.basename(s) + ".o")
            made.append(obj)
            jobs.append([hipcc, *HIPCC_FLAGS, *([] if s in NAN_SOURCES else [NO_NANS]),
                         "-I" + os.path.join(ROOT, "include"), "-c", "-o", obj, os.path.join(HERE, s)])
        with concurrent.futures.ThreadPoolExecutor(len(jobs)) as pool:
            for done in [pool.submit(_run, j, verbose) for j in jobs]:
                done.result()
        _run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *made], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
