"""The host half of the operators around the products under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): tests/sanitize/serving_driver.c
against csrc/mxserve.hip and csrc/mxgemm.hip built for the host alone, with an
empty offload bundle in the kernels' place, so no kernel can start."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_mm_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang"


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)
    assert r.returncode == 0, "%s\n%s%s" % (" ".join(cmd), r.stdout[-3000:], r.stderr[-3000:])
    return r


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="needs ROCm hipcc and clang")
def test_serving_host_code_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libmx_asan.so")
    _run([HIPCC, "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-o", lib, os.path.join(CSRC, "mxserve.hip"), os.path.join(CSRC, "mxgemm.hip")])
    # the symbols the missing device passes would have defined: offload
    # bundles, here empty ones
    syms = [s for s in _run(["nm", "-u", lib]).stdout.split() if s.startswith("__hip_fatbin_")]
    assert syms
    stub = tmp_path / "bundle.c"
    stub.write_text("".join('const char %s[32] __attribute__((aligned(4096))) = "__CLANG_OFFLOAD_BUNDLE__";\n' % s
                            for s in syms))
    exe = str(tmp_path / "serving_asan")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-o", exe,
          os.path.join(ROOT, "tests", "sanitize", "serving_driver.c"), str(stub), "-L" + str(tmp_path), "-lmx_asan",
          "-Wl,-rpath," + str(tmp_path), "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-lm"])
    r = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "serving sanitizer run ok" in r.stdout
