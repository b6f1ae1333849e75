"""Build the gfx950 HIP library in-tree (hipcc cross-compiles without a GPU)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmxgemm.so")
SOURCES = [os.path.join(CSRC, f) for f in ("mxgemm.hip", "mxserve.hip", "mxdraft.hip", "mxmoe.hip")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hpp", ".h"))] + \
    [os.path.join(ROOT, "include", "mxgemm.h")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed FP32 VALU forms stay off: plain scalar float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _depends(obj: str):
    """The files an object was made from (the compiler's own list), or None."""
    try:
        with open(obj[:-2] + ".d") as f:
            words = f.read().replace("\\\n", " ").split()
    except OSError:
        return None
    return [w for w in words if not w.endswith(":")]


def _fresh(obj: str) -> bool:
    deps = _depends(obj)
    if not deps or not os.path.exists(obj):
        return False
    t = os.path.getmtime(obj)
    return all(os.path.exists(d) and os.path.getmtime(d) <= t for d in deps + [__file__])


def build(force: bool = True, verbose: bool = False) -> str:
    """Compile libmxgemm.so, the sources side by side.  Always recompiles
    unless force=False, which keeps every object (and the library) that is
    newer than its sources."""
    if not force and os.path.exists(LIB):
        t = os.path.getmtime(LIB)
        if all(os.path.getmtime(d) <= t for d in DEPS):
            return LIB
    os.makedirs(OBJ, exist_ok=True)
    jobs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, os.path.basename(src)[:-4] + ".o")
        objs.append(obj)
        if not force and _fresh(obj):
            continue
        cmd = [HIPCC] + FLAGS + ["-MD", "-MF", obj[:-2] + ".d", "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = 0
    for obj, p in jobs:
        out = p.communicate()[0]
        if p.returncode != 0:
            sys.stderr.write(out)
            failed = p.returncode
            if os.path.exists(obj):
                os.remove(obj)
    if failed:
        raise RuntimeError("hipcc failed (%d)" % failed)
    tmp = LIB + ".tmp%d" % os.getpid()
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed (%d)" % r.returncode)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--stale" not in sys.argv, verbose=True))
