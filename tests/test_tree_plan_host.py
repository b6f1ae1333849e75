"""Which kernel of mx_tree_attention the inputs of treecases.py take, by the
library's own plan (tests/plan/tree_plan.hip, host code)."""
from __future__ import annotations

import os
import subprocess

import pytest

from tests import treecases as tc
from tests.test_sanitize_serving import HIPCC, ROOT, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs ROCm hipcc")
def test_the_cases_take_the_kernels_that_they_are_named_by(tmp_path):
    exe = str(tmp_path / "tree_plan")
    _run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-o", exe, os.path.join(ROOT, "tests", "plan", "tree_plan.hip")])
    calls = [(dim,) + c for dim in (64, 128) for c in tc.plans()]
    lines = ["%d %d 1 4 %d %d %d %d %d" % (len(seqs), sum(n for n, _ in seqs), dim, page, width, window, most)
             for dim, _, seqs, page, width, window, most in calls]
    r = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=60)
    assert r.returncode == 0
    got = [int(w) for w in r.stdout.split()]
    assert got == [c[1] for c in calls], [(g, c) for g, c in zip(got, calls) if g != c[1]][:5]
    assert {c[1] for c in calls} == {16, 32, 128, 256}
