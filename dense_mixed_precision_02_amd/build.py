"""Build libdmp_gemm.so for gfx950 with hipcc (in-tree)."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

_HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = [os.path.join(_HERE, "csrc", "gemm_api.hip"), os.path.join(_HERE, "csrc", "ragged_api.hip")]
OUT = os.path.join(_HERE, "libdmp_gemm.so")
# The race-check variant: every pipeline step waits for its copies and meets
# every wave; its results must equal the library's bit for bit.
OUT_SYNC = os.path.join(_HERE, "libdmp_gemm_sync.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 VALU forms stay off; the compiler still emits the scalar forms
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(args: list) -> subprocess.Popen:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    return subprocess.Popen([hipcc, *args], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _finish(jobs: list, verbose: bool) -> None:
    failed = []
    for name, proc in jobs:
        _, err = proc.communicate()
        if proc.returncode != 0:
            failed.append(name)
        if proc.returncode != 0 or verbose:
            sys.stderr.write(err)
    if failed:
        raise RuntimeError("hipcc failed for " + ", ".join(failed))


def build(verbose: bool = False) -> str:
    """Builds the library and its race-check variant, every source of both in
    parallel; returns the library's path."""
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as tmp:
        libs = []
        jobs = []
        for out, extra in ((OUT, []), (OUT_SYNC, ["-DDMP_EXTRA_SYNC"])):
            objs = [os.path.join(tmp, os.path.basename(out) + os.path.basename(s) + ".o") for s in SOURCES]
            libs.append((out, objs))
            jobs += [(s, _run([*compile_flags, *extra, "-c", "-o", o, s])) for s, o in zip(SOURCES, objs)]
        _finish(jobs, verbose)
        _finish([(out, _run(["--offload-arch=gfx950", "-shared", "-fPIC", "-o", out + ".tmp", *objs]))
                 for out, objs in libs], verbose)
    for out in (OUT, OUT_SYNC):
        os.replace(out + ".tmp", out)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
