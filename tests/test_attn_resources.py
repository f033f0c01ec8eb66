"""Registers of the attention kernels in the built library (no GPU): the plan deals the
cache out in as many pieces as the chip holds workgroups at once, which it takes from
groups_per_unit; the compiler's kernels have to fit that many, without spills."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from precision_decode_amd import _binding

READELF = shutil.which("llvm-readelf") or "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(data):
    """The gfx950 code objects of the library's offload bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            name = data[entry + 24:entry + 24 + length].decode()
            if "gfx950" in name and size:
                yield data[at + offset:at + offset + size]
            entry += 24 + length
        at = data.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{(name, template arguments): resources} of the attention kernels."""
    if not os.path.exists(READELF):
        pytest.skip("needs llvm-readelf")
    if not os.path.exists(_binding.LIB_PATH):
        from precision_decode_amd import build
        build.build()
    found = {}
    folder = tmp_path_factory.mktemp("objects")
    with open(_binding.LIB_PATH, "rb") as f:
        objects = list(code_objects(f.read()))
    for i, code in enumerate(objects):
        path = str(folder / f"{i}.elf")
        with open(path, "wb") as f:
            f.write(code)
        notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True, check=True).stdout
        for part in notes.split("  - .agpr_count:")[1:]:
            part = ".agpr_count:" + part
            name = re.search(r"\.name:\s+_ZN9nvfp4attn\d+(attn_[a-z_]+?)I((?:Li\d+E)+)E", part)
            if name:
                key = (name[1], tuple(int(n) for n in re.findall(r"Li(\d+)E", name[2])))
                found[key] = {n: int(v) for n, v in re.findall(
                    r"\.(agpr_count|vgpr_count|vgpr_spill_count|private_segment_fixed_size|group_segment_fixed_size):\s+(\d+)",
                    part)}
    return found


def groups_per_unit(dp, rows):
    """As the plan has it."""
    return (5 if dp <= 64 else 4 if dp <= 128 else 2) if rows <= 16 else 3 if dp <= 64 else 2


@pytest.mark.parametrize("name", ["attn_whole", "attn_pieces"])
@pytest.mark.parametrize("blocks,tiles", [(4, 1), (4, 2), (8, 1), (8, 2), (12, 1), (16, 1)])
def test_stream_kernels_fit_their_workgroups(kernels, name, blocks, tiles):
    k = kernels[name, (blocks, tiles)]
    groups = groups_per_unit(16 * blocks, 16 * tiles)
    # a workgroup has a wave on each SIMD, whose 512 registers are given out in eights
    assert -(-(k["vgpr_count"] + k["agpr_count"]) // 8) * 8 * groups <= 512
    assert k["vgpr_spill_count"] == k["private_segment_fixed_size"] == 0
    assert k["group_segment_fixed_size"] * groups <= 160 * 1024


def test_stream_kernels_are_those_of_the_plan(kernels):
    assert {key for key in kernels if key[0] in ("attn_whole", "attn_pieces")} == {
        (name, shape) for name in ("attn_whole", "attn_pieces")
        for shape in ((4, 1), (4, 2), (8, 1), (8, 2), (12, 1), (16, 1))}


@pytest.mark.parametrize("blocks", [4, 8, 12, 16])
@pytest.mark.parametrize("waves", [4, 8])
def test_tile_kernels_fit_two_waves_a_simd(kernels, blocks, waves):
    k = kernels["attn_tiles", (blocks, waves)]
    assert k["vgpr_count"] + k["agpr_count"] <= 256 and k["group_segment_fixed_size"] <= 80 * 1024
    # heads over 192 keep some of their registers in memory, the others none
    assert blocks == 16 or k["vgpr_spill_count"] == k["private_segment_fixed_size"] == 0
