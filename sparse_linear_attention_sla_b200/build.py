"""Build the CUDA library libsla.so (sm_100a) in the package directory.

    python -m sparse_linear_attention_sla_b200.build [--force]

nvcc cross-compiles for sm_100a without a GPU, one process per translation unit. The CUDA runtime is linked
statically so the library loads in any process that has the NVIDIA driver.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsla.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")))


def nvcc_path():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsla.so")
    return cand


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libsla.so if it is missing or older than its sources; return its path."""
    if not force and up_to_date():
        return LIB
    log = os.path.join(PKG, "build.log")
    text = ""
    with tempfile.TemporaryDirectory() as tmp:
        units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
        objects = [os.path.join(tmp, os.path.basename(u) + ".o") for u in units]
        cmds = [[nvcc_path(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", u, "-o", o]
                for u, o in zip(units, objects)]
        procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
        results = [(p.communicate()[0], p.returncode) for p in procs]
        if all(rc == 0 for _, rc in results):
            cmds.append([nvcc_path(), *LINK_FLAGS, *objects, "-o", LIB + ".tmp"])
            res = subprocess.run(cmds[-1], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            results.append((res.stdout, res.returncode))
        for cmd, (out, _) in zip(cmds, results):
            text += " ".join(cmd) + "\n" + out
    with open(log, "w") as f:
        f.write(text)
    rc = max((rc for _, rc in results), key=abs)
    if rc != 0:
        sys.stderr.write(text[-6000:])
        raise RuntimeError(f"nvcc failed (exit {rc}); see {log}")
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print(text)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
