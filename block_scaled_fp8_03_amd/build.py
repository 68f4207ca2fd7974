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


def _written(op: str, args) -> frozenset:
    """The VGPRs that an instruction of the vector ALU writes."""
    if not op.startswith("v_") or op.startswith("v_cmp"):
        return frozenset()
    return frozenset(r for a in args[:2 if "swap" in op else 1] for r in _vgprs(a))


def check_listing(src: str, text: str) -> None:
    """Raises if the listing of a source in OWN_AGPR_SOURCES touches an AGPR
    outside inline assembly, spills, or writes an operand of an MFMA of the
    inline assembly within two instructions or wait states before it (which the
    compiler would see to for its own), on any way there: the two places before
    the start of a block are those before each jump to it, and above it if that falls through."""
    tails = {}                     # label -> VGPRs written in the two places before it, over all ways
    lines = text.splitlines()
    # in the order of the text, until what jumps back bring to earlier labels changes no more
    changed = True
    while changed:
        changed, inside, falls = False, False, False
        before = [frozenset(), frozenset()]

        def reach(label):
            nonlocal changed
            old = tails.get(label, [frozenset(), frozenset()])
            new = [o | w for o, w in zip(old, before)]
            if new != old:
                tails[label], changed = new, True

        for line in lines:
            if "#ASMSTART" in line or "#ASMEND" in line:
                inside = "#ASMSTART" in line
                continue
            label = re.match(r"([.\w$]+):", line)
            if label:
                if falls and label[1].startswith(".L"):
                    reach(label[1])
                before, falls = list(tails.get(label[1], [frozenset(), frozenset()])), True
                continue
            m = re.match(r"\s+([vdsgb]\w*_\w+)\s*(.*)", line.split(";")[0])
            if not m:
                continue
            op, args = m[1], [a.strip() for a in m[2].split(",")]
            if not inside and (re.search(r"(^|[ ,])a(\d|\[)", m[2]) or op.startswith("scratch_")):
                raise RuntimeError(f"{src}: the compiler uses registers that the kernel keeps for itself: {line.strip()}")
            if inside and op.startswith("v_mfma"):
                if {r for a in args[1:3] for r in _vgprs(a)} & (before[0] | before[1]):
                    raise RuntimeError(f"{src}: an operand is written just before its MFMA: {line.strip()}")
            if op == "s_endpgm":
                falls, before = False, [frozenset(), frozenset()]
            elif op.startswith(("s_branch", "s_cbranch")):
                before = [before[1], frozenset()]
                reach(args[0])
                if op == "s_branch":
                    falls, before = False, [frozenset(), frozenset()]
                else:
                    falls = True
            elif op.startswith(("s_setpc", "s_swappc", "s_call")):
                raise RuntimeError(f"{src}: a jump whose target the check does not follow: {line.strip()}")
            else:
                n = min(int(args[0], 0) + 1, 2) if op == "s_nop" else 1
                before = (before + [frozenset()] * n if op == "s_nop" else before + [_written(op, args)])[-2:]
                falls = True


def compile_listed(cmd, src: str, build_dir: str):
    """(object, device listing) of one compilation."""
    name = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    _run([*cmd, "-c", src, "-o", obj, "-save-temps=obj"])
    with open(os.path.join(build_dir, f"{name}-hip-amdgcn-amd-amdhsa-gfx950.s")) as f:
        return obj, f.read()


def _run(cmd) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")


def _compile(src: str, build_dir: str) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(build_dir, src + ".o")
    if src.endswith(".cpp"):
        _run([HIPCC, *COMMON_FLAGS, "--offload-arch=gfx950", "-c", path, "-o", obj])
        return obj
    own = OWN_AGPR_FLAGS if src in OWN_AGPR_SOURCES else []
    form = [] if src in AGPR_SOURCES else VGPR_FORM
    cmd = [HIPCC, *COMMON_FLAGS, *HIP_FLAGS, *form, *own, "-x", "hip"]
    if own:
        obj, text = compile_listed(cmd, path, build_dir)
        check_listing(src, text)
    else:
        _run([*cmd, "-c", path, "-o", obj])
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
