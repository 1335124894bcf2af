"""Build the HIP library in-tree with hipcc for gfx950.

``python -m draft_verify_sampling_spec_amd.build`` (or ``build_library()``)
compiles ``csrc/spec_verify.hip`` (verification), ``csrc/budget_schedule.hip``
(the verify-budget scheduler), ``csrc/head_stats.hip`` (output-head row
statistics), ``csrc/verify_hidden.hip`` (verification from hidden states),
``csrc/markov_draft.hip`` (the drafter's low-rank Markov head),
``csrc/block_cache.hip`` (the paged 4-bit key/value cache),
``csrc/page_tables.hip`` (its page tables from the requests' lengths),
``csrc/rotate_write.hip`` (normalised and rotated heads on their way into it),
``csrc/block_attention.hip`` (attention of drafted blocks over it),
``csrc/sink_attention.hip`` (under a window with sink tokens),
``csrc/shared_attention.hip`` (for requests that share a prefix) and
``csrc/head_fp8.hip`` (the output head in 8-bit floating point) into
``libspec_verify.so`` next to this file.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRC = os.path.join(PKG_DIR, "csrc", "spec_verify.hip")
SOURCES = [SRC, os.path.join(PKG_DIR, "csrc", "budget_schedule.hip"),
           os.path.join(PKG_DIR, "csrc", "head_stats.hip"),
           os.path.join(PKG_DIR, "csrc", "verify_hidden.hip"),
           os.path.join(PKG_DIR, "csrc", "markov_draft.hip"),
           os.path.join(PKG_DIR, "csrc", "block_cache.hip"),
           os.path.join(PKG_DIR, "csrc", "page_tables.hip"),
           os.path.join(PKG_DIR, "csrc", "rotate_write.hip"),
           os.path.join(PKG_DIR, "csrc", "block_attention.hip"),
           os.path.join(PKG_DIR, "csrc", "sink_attention.hip"),
           os.path.join(PKG_DIR, "csrc", "shared_attention.hip"),
           os.path.join(PKG_DIR, "csrc", "head_fp8.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libspec_verify.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
# A test helper (not part of the library): a bounded kernel that holds CUs.
TEST_SRC = os.path.join(ROOT, "tests", "occupy_kernel.hip")
TEST_LIB_PATH = os.path.join(ROOT, "tests", "libsv_occupy.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def compile_command(out: str, sources, *flags) -> list:
    return [
        hipcc(),
        f"--offload-arch={ARCH}",
        "-O3",
        "-std=c++17",
        "-fPIC",
        *flags,
        # Floating-point expressions are evaluated as written (no FMA
        # contraction), so identical expressions give identical values.
        "-ffp-contract=off",
        # Keep the compiler from emitting packed fp32 VALU instructions.
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall",
        "-I", INCLUDE,
        *sources,
        "-o", out,
    ]


def build_library(verbose: bool = True) -> str:
    """Compile the library and the tests' helper (always; outputs are
    replaced atomically). The sources are compiled side by side."""
    if os.path.exists(TEST_SRC):
        _compile(compile_command(TEST_LIB_PATH + ".tmp", [TEST_SRC], "-shared"), verbose)
        os.replace(TEST_LIB_PATH + ".tmp", TEST_LIB_PATH)
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _compile(compile_command(so[1], [so[0]], "-c"), verbose),
                          zip(SOURCES, objects)))
        _compile([hipcc(), f"--offload-arch={ARCH}", "-shared", *objects, "-o", LIB_PATH + ".tmp"],
                 verbose)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)
    return LIB_PATH


def _compile(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}")
    if verbose and res.stderr.strip():
        # Warnings (the host pass does not know the packed-fp32 feature flag).
        lines = [l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l]
        if any(l.strip() for l in lines):
            sys.stderr.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    build_library()
