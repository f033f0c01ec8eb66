"""Linear-layer cases with the kernel that the plan gives them: the GPU tests run
them, and a CPU test checks that the plan still gives them that kernel, so that
a change of the plan's times cannot empty the tests."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (n, m, k, gated): the tile shape (rows of each matrix x tokens) and the parts of K.  k is no
# multiple of 64, m none of 8.
TILES = {
    (130, 1030, 336, False): "tile 64x32 1", (100, 4100, 336, False): "tile 64x64 1",
    (513, 2050, 336, False): "tile 128x64 1", (1025, 2050, 592, False): "tile 128x128 1",
    (1025, 4100, 336, False): "tile 256x128 1", (2100, 4100, 336, False): "tile 256x256 1",
    (130, 1030, 592, True): "tile 64x32 1", (100, 4100, 336, True): "tile 64x64 1",
    (513, 2050, 592, True): "tile 64x128 1", (1025, 2050, 336, True): "tile 128x128 1",
    (1025, 4100, 336, True): "tile 128x256 1",
}
SPLIT_TILES = {
    (97, 2050, 8208, False): "tile 128x64 4", (130, 1030, 8208, False): "tile 128x64 8",
    (385, 518, 8208, False): "tile 64x64 4", (17, 2050, 8208, False): "tile 64x32 4",
    (130, 1030, 4112, True): "tile 64x64 4", (70, 2050, 4112, True): "tile 64x32 2",
    (97, 2050, 8208, True): "tile 64x128 4", (97, 1030, 16400, True): "tile 64x128 8",
}
# k of whole rows of 64: special values, epilogues, tails of the activations, far rows
WHOLE_TILES = {
    (130, 1030, 320, False): "tile 64x32 1", (130, 1030, 320, True): "tile 64x32 1",
    (513, 2050, 320, False): "tile 128x64 1", (513, 2050, 320, True): "tile 64x128 1",
    (1025, 4100, 320, False): "tile 256x128 1", (1025, 4100, 320, True): "tile 128x256 1",
    (300, 2050, 64, False): "tile 64x64 1", (2100, 4100, 64, False): "tile 256x256 1",
}


def printer(folder):
    """The program that prints plans, built in that folder."""
    exe = os.path.join(str(folder), "ffn_plan_print")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "precision_decode_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "ffn_plan_print.cpp"), "-o", exe], check=True)
    return exe


def plans(exe, lines):
    res = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout.splitlines()


have_compiler = shutil.which("g++") is not None
