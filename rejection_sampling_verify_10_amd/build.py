"""Builds libspecverify.so (the C-ABI HIP library) for gfx950, in-tree.

    python -m rejection_sampling_verify_10_amd.build
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
if __package__:
    from .waits import unwaited
else:
    sys.path.insert(0, HERE)
    from waits import unwaited
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libspecverify.so")
SOURCES = ["alpha.hip", "api.hip", "dense_tr.hip", "dense_walk.hip", "eagle2.hip", "kv_commit.hip", "kvq_append.hip",
           "kvq_attention.hip", "kvq_evict.hip", "kvq_score.hip", "lmhead.hip", "logprob.hip", "nucleus.hip", "paged_append.hip", "paged_attention.hip",
           "paged_plan.hip", "paged_step.hip", "rowstats.hip",
           "topk.hip", "tree_cluster.hip", "tree_sample.hip", "verify.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# Matrix products in inline assembly: what the compiler made of these is looked over for the waits that it does not place.
OWN_WAITS = ("paged_attention.hip",)

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 VALU forms stay off: plain float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def check_waits(src: str, assembly: str) -> None:
    """Raises if a kernel of `src` reads a product's sums too early, or has none of the products that were to be looked over."""
    with open(assembly) as f:
        found, early = unwaited(f.read())
    if early or not found:
        raise RuntimeError(f"{src}: {found} matrix products in assembly, accesses of their sums that wait too little: {early[:5]}")


def build(verbose: bool = False) -> str:
    """Compile every source and link the shared library; returns its path."""
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if src in OWN_WAITS:
            cmd.append("--save-temps=obj")
        r = subprocess.run(cmd, capture_output=True, text=True)
        msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                        if "packed-fp32-ops" not in l and l.strip())
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
        if verbose and msg:
            print(msg, file=sys.stderr)
        if src in OWN_WAITS:
            check_waits(src, os.path.join(objdir, src.replace(".hip", "-hip-amdgcn-amd-amdhsa-gfx950.s")))
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
