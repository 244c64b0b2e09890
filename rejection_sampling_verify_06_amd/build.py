"""Build the HIP library (libspec_verify.so) in-tree for gfx950 with hipcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_NAME = "libspec_verify.so"
SOURCES = ["csrc/sv_kernels.hip", "csrc/sv_ngram.hip", "csrc/sv_stats.hip", "csrc/sv_filter.hip", "csrc/sv_noalloc.hip",
           "csrc/sv_logprobs.hip", "csrc/sv_attention.hip", "csrc/sv_attention_e4m3.hip", "csrc/sv_attention_int8.hip",
           "csrc/sv_attention_shared.hip", "csrc/sv_attention_shared_e4m3.hip", "csrc/sv_attention_shared_int8.hip", "csrc/sv_cache.hip", "csrc/sv_rope.hip", "csrc/sv_api.cpp", "csrc/sv_serving_api.cpp"]
ARCH = "gfx950"


def library_path() -> str:
    return os.path.join(HERE, LIB_NAME)


def hipcc_command(source: str, out: str) -> list:
    """The compilation of one source."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return [
        hipcc, f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
        # packed fp32 instructions are kept out of every kernel
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        # no implicit a*b+c fusion: the softmax merge relies on round(m*c) being
        # the same value wherever it is formed; fusion is written out as fmaf
        "-ffp-contract=off",
        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
        os.path.join(HERE, source), "-o", out,
    ]


def link_command(objects: list, out: str) -> list:
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return [hipcc, f"--offload-arch={ARCH}", "-fPIC", "-shared", *objects, "-o", out]


def _run(cmd: list, verbose: bool):
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = [l for l in (r.stderr or "").splitlines() if "packed-fp32-ops" not in l and l.strip()]
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(noise))
    if verbose and noise:
        print("\n".join(noise))


def build_library(verbose: bool = False) -> str:
    """Compile the library, its sources side by side; returns its path.  Links
    to a temporary name and renames, so a concurrent loader never sees a
    half-written file."""
    out = library_path()
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory(prefix="spec_verify_") as work:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        jobs = [hipcc_command(s, o) for s, o in zip(SOURCES, objects)]
        if verbose:
            print(" ".join(jobs[0]) + f"    (and {len(jobs) - 1} more sources)", flush=True)
        # one compiler a CPU; two at least, since the largest source takes half of the time
        with ThreadPoolExecutor(max(2, min(len(jobs), os.cpu_count() or 2, 8))) as pool:
            for _ in pool.map(lambda c: _run(c, verbose), jobs):
                pass
        _run(link_command(objects, tmp), verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build_library(verbose=True))
