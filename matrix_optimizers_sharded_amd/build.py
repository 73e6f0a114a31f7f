"""Build libmatopt.so in-tree for gfx950 with hipcc (cross-compiles without a GPU).

    python -m matrix_optimizers_sharded_amd.build [--verbose]
"""

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
# one translation unit per group of entry points, compiled side by side
SOURCES = sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))
LIB = os.path.join(PKG, "lib", "libmatopt.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def build(verbose=False, extra=()):
    where = os.path.dirname(LIB)
    os.makedirs(where, exist_ok=True)
    t0 = time.time()
    # a folder of its own, so that builds at once do not share files
    with tempfile.TemporaryDirectory(prefix="build-", dir=where) as tmp:
        def compile_one(src):
            name = os.path.splitext(os.path.basename(src))[0]
            obj = os.path.join(tmp, name + ".o")
            # the unit's id in the code, which the compiler would make from the paths: the
            # same sources have to give the same code wherever they are
            cmd = [HIPCC, *FLAGS, *extra, f"-cuid={name}", "-c", "-o", obj, src]
            return obj, subprocess.run(cmd, capture_output=True, text=True)

        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            done = list(pool.map(compile_one, SOURCES))
        results = [r for _, r in done]
        lib = os.path.join(tmp, os.path.basename(LIB))
        if all(r.returncode == 0 for r in results):
            link = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-o", lib, *[o for o, _ in done]]
            results.append(subprocess.run(link, capture_output=True, text=True))
        log = [r.stdout + r.stderr for r in results]
        if any(r.returncode != 0 for r in results):
            sys.stderr.write("".join(log))
            raise RuntimeError("hipcc failed building libmatopt.so")
        os.replace(lib, LIB)
    if verbose:
        sys.stderr.write("".join(log))
        print(f"built {LIB} in {time.time() - t0:.1f}s")
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv)
