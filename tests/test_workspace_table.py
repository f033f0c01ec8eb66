"""The table of library-owned workspaces (``tests/host/workspace_check.cpp``)
under the address and undefined-behaviour sanitizers.  No GPU."""
import os
import shutil

import pytest

from test_host_sanitized import HOST, ROOT, SAN, build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_workspace_table_under_sanitizers(tmp_path):
    exe = str(tmp_path / "workspace_check")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "precision_decode_amd", "csrc"),
           os.path.join(HOST, "workspace_check.cpp"), "-o", exe]
    run = build_and_run(cmd, exe)
    assert run.returncode == 0 and "workspace_check ok" in run.stdout, run.stdout + run.stderr


def test_no_other_container_in_the_c_entry_points():
    """What could throw behind a C entry point is in the table, which lets nothing out."""
    csrc = os.path.join(ROOT, "precision_decode_amd", "csrc")
    for name in os.listdir(csrc):
        if name != "workspace_table.h":
            with open(os.path.join(csrc, name)) as f:
                text = f.read()
            for word in ("std::map", "std::vector", "std::string", "std::unordered", "std::function", "throw "):
                assert word not in text, f"{name}: {word}"
