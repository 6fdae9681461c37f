"""Build libpn.so (the HIP kernels and the C ABI of include/pn.h) for gfx950 with hipcc."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libpn.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 (v_pk_*_f32) is kept out of generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))


def build(out: str = LIB, verbose: bool = False) -> str:
    """Compile every source (up to eight at once) and link them into `out`."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        msgs = [l for l in (r.stdout + r.stderr).splitlines()
                if "packed-fp32-ops" not in l or "error" in l]
        if r.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
        if verbose and msgs:
            print("\n".join(msgs))

    with tempfile.TemporaryDirectory() as tmp:
        jobs = []
        for src in sources():
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            jobs.append((obj, [hipcc, *HIPCC_FLAGS, "-c", "-I", os.path.join(ROOT, "include"),
                               "-I", os.path.join(HERE, "csrc"), src, "-o", obj]))
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(run, [cmd for _, cmd in jobs]))
        run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", *[obj for obj, _ in jobs], "-o",
             out + ".tmp"])
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
