"""The feed-forward operators' host plan at the largest sizes of its shape
rules (``tests/host/ffn_limits_check.cpp``), built with g++ under the address
and undefined-behaviour sanitizers.  No GPU."""
import os
import shutil

import pytest

from test_host_sanitized import HOST, ROOT, SAN, build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_ffn_limits_under_sanitizers(tmp_path):
    exe = str(tmp_path / "ffn_limits_check")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "precision_decode_amd", "csrc"),
           os.path.join(HOST, "ffn_limits_check.cpp"), "-o", exe]
    run = build_and_run(cmd, exe)
    assert run.returncode == 0 and "ffn_limits_check ok" in run.stdout, run.stdout + run.stderr
