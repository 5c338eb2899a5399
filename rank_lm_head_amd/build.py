"""Builds liblrhead.so (and the benchmark's read probe, libprobe.so) in-tree
with hipcc for gfx950.

    python -m rank_lm_head_amd.build

Cross-compiles without a GPU. Each source becomes an object of its own, the
objects are compiled in parallel and then linked into the shared library.
Packed fp32 instructions are disabled for the device code; hipcc's host pass
warns that it does not know that feature, which is harmless. The device
assembly of each source is looked through for a mistake of the compiler (see
lost_lanes); a source that has it is not built.
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "liblrhead.so")
PROBE_LIB = os.path.join(PKG, "libprobe.so")   # measurement only, not the head's ABI
PROBE_SOURCE = "probe_read.hip"
OBJ = os.path.join(PKG, "_build")
SOURCES = ["kernels_small.hip", "kernels_mfma.hip", "kernels_gemm.hip", "kernels_merge.hip", "kernels_branch.hip",
           "kernels_factor.hip", "kernels_b1.hip", "kernels_distill.hip", "kernels_beam.hip", "kernels_sample.hip",
           "kernels_embed.hip", "lrhead.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Werror=return-type", "-Werror=infinite-recursion",
]
NOISE = "is not a recognized feature for this target"


def _run(cmd: list[str]) -> tuple[int, list[str]]:
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if NOISE not in ln]
    return res.returncode, msgs


_SKIP = re.compile(r"\s*s_cbranch_execz\s+(\S+)")
_LABEL = re.compile(r"(\.L\S+|_Z\w+):")
_REJOIN = re.compile(r"s_or_b64 exec, exec,|s_or_saveexec_b64 ")
_EXEC = re.compile(r"s_\w+ exec,|s_\w+saveexec")
_VECTOR = re.compile(r"(v_(?!readlane|readfirstlane|writelane|cmp)|ds_|global_|flat_|buffer_|scratch_)")


def lost_lanes(asm: str) -> list[str]:
    """Vector instructions at the head of a block to which lanes skip, in front
    of the instruction that brings those lanes back.

    The compiler's register allocator makes copies of registers at the heads of
    blocks. Where a scalar copy already stands in front of the lanes' return,
    it has put a vector copy (or a spill) there as well: of the lanes that
    skipped, nothing is copied, and a copy back later leaves garbage in them. A
    build of sample_rows_kernel whose registers were a few short lost its lane
    numbers this way, and read outside its memory. Code of the sources' own
    does not stand there: a block to which lanes skip begins with their return.
    """
    lines = asm.split("\n")
    skipped_to = {m.group(1) for m in map(_SKIP.match, lines) if m}
    found, kernel, head, vector = [], "", False, []
    for number, line in enumerate(lines, 1):
        m = _LABEL.match(line)
        if m:
            kernel = m.group(1) if m.group(1).startswith("_Z") else kernel
            head, vector = m.group(1) in skipped_to, []
            continue
        text = line.split(";")[0].strip()
        if not head or not text or text.startswith("."):
            continue
        if _REJOIN.match(text):
            found += [f"{kernel}, line {n}: {t}" for n, t in vector]
            head = False
        elif _EXEC.match(text) or text.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            head = False
        elif _VECTOR.match(text):
            vector.append((number, text))
    return found


def _compile(source: str, obj: str) -> tuple[int, list[str]]:
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with tempfile.TemporaryDirectory(dir=OBJ) as room:
        tmp = os.path.join(room, os.path.basename(obj))
        cmd = [HIPCC, *FLAGS, *inc, "-save-temps=obj", "-c", source, "-o", tmp]
        rc, msgs = _run(cmd)
        if rc != 0:
            return rc, [" ".join(cmd), *msgs]
        asm = glob.glob(os.path.join(room, "*gfx950*.s"))
        if not asm:
            return 1, [f"{source}: no device assembly to look through"]
        lost = [x for path in asm for x in lost_lanes(open(path).read())]
        if lost:
            return 1, [f"{source}: compiled so that lanes lose registers", *lost]
        os.replace(tmp, obj)
    return 0, msgs


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    jobs = [(os.path.join(CSRC, s), os.path.join(OBJ, os.path.splitext(s)[0] + ".o")) for s in SOURCES]
    probe_tmp = PROBE_LIB + ".tmp"
    probe = [HIPCC, *FLAGS, "-shared", os.path.join(CSRC, PROBE_SOURCE), "-o", probe_tmp]
    workers = max(1, min(len(jobs), int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))
    with ThreadPoolExecutor(max_workers=workers) as ex:
        probe_job = ex.submit(_run, probe)
        results = list(ex.map(lambda j: _compile(*j), jobs))
        probe_res = probe_job.result()
    if probe_res[0] != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(probe) + "\n" + "\n".join(probe_res[1]))
    os.replace(probe_tmp, PROBE_LIB)
    out = []
    for rc, msgs in results:
        if rc != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        out += msgs
    tmp = LIB + ".tmp"
    link = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *[obj for _, obj in jobs], "-o", tmp]
    rc, msgs = _run(link)
    if rc != 0:
        raise RuntimeError("link failed:\n" + " ".join(link) + "\n" + "\n".join(msgs))
    out += msgs
    if verbose and out:
        print("\n".join(out), file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
