"""Build the CUDA library in-tree: async_rl_b200/libbi_isloss.so (sm_100a only).

    python -m async_rl_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbi_isloss.so")
SOURCES = ["bi_api.cu", "bi_rope.cu", "bi_adamw.cu", "bi_attn.cu"]
HEADERS = ["host.h", "sm100.cuh", "kernels_lm.cuh", "kernels_decode.cuh", "kernels_dw.cuh", "kernels_model.cuh",
           "kernels_small.cuh", "kernels_rope.cuh", "kernels_adamw.cuh", "kernels_attn.cuh",
           "kernels_attn_bwd.cuh"]
PUBLIC = ["bi_isloss.h", "bi_model.h", "bi_optim.h"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", h) for h in PUBLIC]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _run(cmd) -> str:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + proc.stdout + proc.stderr)
    return proc.stdout + proc.stderr


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compiles the sources side by side and links them."""
    if not force and not needs_build():
        return LIB
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "-I" + os.path.join(ROOT, "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    nvcc = nvcc_path()
    with tempfile.TemporaryDirectory(prefix="bi_build_") as tmp:
        objs = [os.path.join(tmp, f + ".o") for f in SOURCES]
        cmds = [[nvcc, *flags, "-c", "-o", o, os.path.join(CSRC, f)] for f, o in zip(SOURCES, objs)]
        with concurrent.futures.ThreadPoolExecutor(len(cmds)) as pool:
            said = list(pool.map(_run, cmds))
        if ptxas_verbose:
            sys.stderr.write("".join(said))
        _run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", LIB + ".tmp", *objs])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
