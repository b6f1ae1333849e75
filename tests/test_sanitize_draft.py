"""The host half of the operators for drafted tokens and for experts under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
tests/sanitize/draft_driver.c against csrc/mxdraft.hip, csrc/mxmoe.hip and what
they call, built for the host alone, with empty offload bundles in the kernels'
place, so no kernel can start."""
from __future__ import annotations

import os

import pytest

from tests.test_sanitize_serving import CLANG, CSRC, HIPCC, ROOT, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="needs ROCm hipcc and clang")
def test_draft_host_code_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libmx_asan.so")
    _run([HIPCC, "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-o", lib] + [os.path.join(CSRC, f) for f in ("mxdraft.hip", "mxmoe.hip", "mxgemm.hip")])
    syms = [s for s in _run(["nm", "-u", lib]).stdout.split() if s.startswith("__hip_fatbin_")]
    assert syms
    stub = tmp_path / "bundle.c"
    stub.write_text("".join('const char %s[32] __attribute__((aligned(4096))) = "__CLANG_OFFLOAD_BUNDLE__";\n' % s
                            for s in syms))
    exe = str(tmp_path / "draft_asan")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-o", exe,
          os.path.join(ROOT, "tests", "sanitize", "draft_driver.c"), str(stub), "-L" + str(tmp_path), "-lmx_asan",
          "-Wl,-rpath," + str(tmp_path), "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-lm"])
    r = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "draft sanitizer run ok" in r.stdout and "runtime error" not in r.stderr, r.stderr[-2000:]
