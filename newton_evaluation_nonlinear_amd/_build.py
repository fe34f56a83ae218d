"""Compile libpn.so in-tree for gfx950 with hipcc.

    python -m newton_evaluation_nonlinear_amd._build

Each source is compiled to an object in parallel (the device code of every
file is self-contained) and its assembly is checked (lost_lanes), then the
objects are linked into libpn.so; the
ceiling microbenchmarks (pn_ceiling.hip) become libpn_ceiling.so.
"""

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpn.so")
# the ceiling microbenchmarks (a measurement tool, include/pn_ceiling.h)
CEILING_LIB = os.path.join(HERE, "libpn_ceiling.so")
CEILING_SOURCES = ["pn_ceiling.hip"]

SOURCES = ["pn_api.cpp", "pn_diag.hip", "pn_cell.hip", "pn_dense.hip", "pn_scan.hip", "pn_static.hip", "pn_small.hip",
           "pn_seq_api.cpp", "pn_rotary.hip", "pn_linattn.hip", "pn_linattn_bf16.hip",
           "pn_linattn_f16.hip", "pn_linattn_f32.hip"]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 ALU forms stay off: keep every FP32 op scalar
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-result",
]


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("hipcc failed building libpn.so")
    return r.stderr


def lost_lanes(asm):
    """Kernels in gfx950 assembly (its lines) that save a register to scratch after a branch on lanes, in the block where they
    meet, before the mask of all lanes is restored: the compiler has done so, and the other lanes then read back garbage."""
    found, name, saved = [], "", False
    for line in asm:
        code = line.split(";")[0].split()
        if line.startswith("_Z"):
            name, saved = line.split(":")[0], False
        elif line.startswith(".LBB") or "; %bb." in line or code and code[0].startswith(("s_cbranch", "s_branch", "s_endpgm")):
            saved = False
        elif code and code[0].startswith("scratch_store"):
            saved = True
        elif saved and code and code[0] == "s_or_b64" and code[1:3] == ["exec,", "exec,"]:
            found.append(name)
            saved = False
    return found


def check_lanes(folder):
    """Raise if assembly files of ``folder`` hold such kernels."""
    for path in sorted(glob.glob(os.path.join(folder, "*gfx950.s"))):
        with open(path) as f:
            found = lost_lanes(f)
        if found:
            raise RuntimeError(f"{os.path.basename(path)}: registers saved under a narrowed lane mask in {', '.join(found)}; "
                               "write the branch on the thread index before it without a branch")


def build(verbose=False):
    with tempfile.TemporaryDirectory(prefix="pn_build_") as tmpd:
        objs, cmds = [], []
        for src in SOURCES:
            obj = os.path.join(tmpd, src + ".o")
            objs.append(obj)
            # the assembly is kept beside the object for check_lanes()
            cmds.append([hipcc()] + FLAGS + ["--save-temps=obj", "-I", os.path.join(ROOT, "include"), "-c",
                                             os.path.join(CSRC, src), "-o", obj])
        cobjs = []
        for src in CEILING_SOURCES:
            obj = os.path.join(tmpd, src + ".o")
            cobjs.append(obj)
            cmds.append([hipcc()] + FLAGS + ["-I", os.path.join(ROOT, "include"), "-c",
                                             os.path.join(CSRC, src), "-o", obj])
        workers = min(len(cmds), max(1, (os.cpu_count() or 1)))
        with ThreadPoolExecutor(max_workers=workers) as ex:
            logs = list(ex.map(_run, cmds))
        check_lanes(tmpd)
        tmp = LIB + ".tmp"
        logs.append(_run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs))
        ctmp = CEILING_LIB + ".tmp"
        logs.append(_run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", ctmp] + cobjs))
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
        for lg in logs:
            lines = [ln for ln in lg.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
            if lines:
                sys.stderr.write("\n".join(lines) + "\n")
    os.replace(tmp, LIB)
    os.replace(ctmp, CEILING_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
