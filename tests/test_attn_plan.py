"""``tests/host/attn_plan_check.cpp`` compiles the plan of the attention operators
(``precision_decode_amd/csrc/attn_plan.h``: shape and stride rules, kernel choice,
workspace layout) with g++ under the address and undefined-behaviour sanitizers and
checks 200000 random shapes against what the kernels assume (no GPU)."""
import os
import shutil

import pytest

from test_host_sanitized import HOST, ROOT, SAN, build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_attn_plan_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_plan_check")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "precision_decode_amd", "csrc"),
           os.path.join(HOST, "attn_plan_check.cpp"), "-o", exe]
    run = build_and_run(cmd, exe)
    assert run.returncode == 0 and "attn_plan_check ok" in run.stdout, run.stdout + run.stderr
