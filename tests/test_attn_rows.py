"""``tests/host/attn_rows_check.cpp`` compiles the launches of norms, cache writes and
cache reads (``precision_decode_amd/csrc/attn_plan.h``) with g++ under the address and
undefined-behaviour sanitizers and checks 300000 shapes up to the borders of the rules:
launches below 2^32 threads that cover every row (no GPU)."""
import os
import shutil

import pytest

from test_host_sanitized import HOST, ROOT, SAN, build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_row_launches_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_rows_check")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "precision_decode_amd", "csrc"),
           os.path.join(HOST, "attn_rows_check.cpp"), "-o", exe]
    run = build_and_run(cmd, exe)
    assert run.returncode == 0 and "attn_rows_check ok" in run.stdout, run.stdout + run.stderr
