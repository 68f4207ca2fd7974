"""Build libfp8bs.so (gfx950) in-tree with hipcc.

Usage: python -m block_scaled_fp8_03_amd.build   (or build() from Python)

Every HIP source is compiled for gfx950 only, with packed-FP32 instructions
disabled and floating-point contraction off (the kernels write every FMA they
want explicitly), then linked into one shared library next to this file.
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfp8bs.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["quant.hip", "gemm.hip", "gemm_e8.hip", "moe_dispatch.hip", "mla.hip",
           "mla_attention.hip", "mla_cache.hip", "abi.cpp"]

COMMON_FLAGS = [
    "-std=c++17", "-O3", "-fPIC", "-Wall", "-Wno-unused-function",
    "-ffp-contract=off",
    f"-I{INCLUDE}", f"-I{CSRC}",
]
HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
# MFMA results in VGPRs: the per-K-block scale fold reads them with VALU FMAs,
# which cannot take AGPR operands.  gemm_e8.hip has no fold and keeps its 256
# accumulators per lane in AGPRs, so it is built without this.
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
AGPR_SOURCES = {"gemm_e8.hip"}
# mla_attention.hip names its accumulator AGPRs in inline assembly; a build in
# which the compiler uses AGPRs (or memory) for anything of its own is refused.
OWN_AGPR_SOURCES = {"mla_attention.hip"}
OWN_AGPR_FLAGS = ["-mllvm", "-amdgpu-spill-vgpr-to-agpr=0"]


def _vgprs(operand: str) -> range:
    """The VGPRs that an operand of a listing names (``v7``, ``v[4:7]``); empty for others."""
    m = re.fullmatch(r"v(\d+)|v\[(\w+):(\w+)\]", operand.strip())
    if not m:
        return range(0)
    return range(int(m[1]), int(m[1]) + 1) if m[1] else range(int(m[2], 0), int(m[3], 0) + 1)


def check_listing(src: str, text: str) -> None:
    """Raises if the listing of a source in OWN_AGPR_SOURCES touches an AGPR
    outside inline assembly, spills, or writes an operand of an MFMA of the
    inline assembly within two instructions or wait states before it (which the
    compiler would see to for its own)."""
    inside, before = False, []
    for line in text.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inside = "#ASMSTART" in line
            continue
        m = re.match(r"\s+([vdsgb]\w*_\w+)\s+(.*)", line.split(";")[0])
        if not m:
            continue
        op, args = m[1], [a.strip() for a in m[2].split(",")]
        if not inside and (re.search(r"(^|[ ,])a(\d|\[)", m[2]) or op.startswith("scratch_")):
            raise RuntimeError(f"{src}: the compiler uses registers that the kernel keeps for itself: {line.strip()}")
        if inside and op.startswith("v_mfma"):
            read = {r for a in args[1:3] for r in _vgprs(a)}
            if any(read & set(w) for w in before[-2:]):
                raise RuntimeError(f"{src}: an operand is written just before its MFMA: {line.strip()}")
        if op == "s_nop":
            before += [range(0)] * (int(args[0], 0) + 1)
        else:
            before.append(_vgprs(args[0]) if op.startswith("v_") and not op.startswith("v_cmp") else range(0))


def _listing(cmd, src: str) -> str:
    res = subprocess.run([*cmd, "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", "-"], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {src}\n{res.stderr}")
    return res.stdout


def _compile(src: str, build_dir: str) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    form = [] if src in AGPR_SOURCES else VGPR_FORM
    own = OWN_AGPR_FLAGS if src in OWN_AGPR_SOURCES else []
    cmd = [HIPCC, *COMMON_FLAGS, *HIP_FLAGS, *form, *own, "-x", "hip"]
    if own:
        check_listing(src, _listing(cmd, src))
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [HIPCC, *COMMON_FLAGS, "--offload-arch=gfx950", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, build_dir), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
