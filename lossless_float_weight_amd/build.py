"""Builds libzn.so in-tree with hipcc for gfx950 (no JIT cache, no pip install)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libzn.so")
SOURCES = ["zn_api.hip", "zn_encode.hip", "zn_decode.hip", "zn_setup.hip", "zn_mx_api.hip", "zn_mx.hip", "zn_mxmm.hip",
           "zn_kv_api.hip", "zn_kv.hip", "zn_attn.hip", "zn_attn_tall.hip"]
ARCH = os.environ.get("ZN_OFFLOAD_ARCH", "gfx950")
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         # packed FP32 instructions are kept out of every kernel
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", os.path.join(HERE, "..", "include")]


# Kernels whose memory instructions the compiler does not see (copies to LDS in
# assembly, waited for by their number) must keep every register: a form of
# them that spilled has given a wrong sum, for a reason that was not found.
NO_SPILLS = {"zn_mxmm.hip": "k_mx_tiled"}
_REMARK = "[-Rpass-analysis=kernel-resource-usage]"


def spilling(report: str, kernel: str) -> list[str]:
    """Instances of `kernel` that spill, from the compiler's report of
    resources; an error if the report names none at all."""
    name, seen, bad = "", 0, []
    for line in report.splitlines():
        m = re.search(r"remark:\s*(.*?):\s*(\S+)", line)
        if m is None or _REMARK not in line:
            continue
        if m[1] == "Function Name":
            name = m[2]
            seen += kernel in name
        elif kernel in name and m[1] in ("ScratchSize [bytes/lane]", "SGPRs Spill", "VGPRs Spill") and m[2] != "0":
            bad.append(f"{name}: {m[1]} {m[2]}")
    if not seen:
        raise RuntimeError(f"the compiler reports no kernel {kernel}")
    return bad


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, src.replace(".hip", ".o"))
    kernel = NO_SPILLS.get(src)
    report = ["-Rpass-analysis=kernel-resource-usage", "-fno-caret-diagnostics"] if kernel else []
    cmd = ["hipcc", *FLAGS, *report, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    errs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l and _REMARK not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{errs}")
    if kernel:
        bad = spilling(r.stderr, kernel)
        if bad:
            raise RuntimeError(f"{src}: registers spill:\n" + "\n".join(bad))
    if errs:
        print(errs, file=sys.stderr)
    return obj


def build() -> str:
    """Compiles every HIP source and links libzn.so; always rebuilds."""
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    r = subprocess.run(["hipcc", "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
