"""Accesses of the mixture-of-experts kernels, modelled on the CPU: ``tests/native/moe_bounds_check.cpp``
evaluates the offset functions that the kernels call (``csrc/moe_offsets.hpp``) over widths of one
block to many and checks that none leaves its operand, and that every block is taken once."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_02_amd", "csrc")
FAMILIES = ("weights", "activations", "staged", "h", "tiles")


def _run(folder, first=CSRC):
    exe = os.path.join(folder, "moe_bounds_check")
    cmd = ["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17", "-I", str(first), "-I", CSRC,
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "moe_bounds_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    found = {}
    for line in r.stdout.splitlines():
        family, _, n, _, v = line.split()
        found[family] = int(n), int(v)
    return found, r.stderr


def test_no_access_leaves_its_operand(tmp_path):
    found, err = _run(str(tmp_path))
    assert set(found) == set(FAMILIES)
    for family, (n, v) in found.items():
        assert n > 1000 and v == 0, (family, n, v, err)


@pytest.mark.parametrize("family, was, planted", [
    ("weights", "(lane >> 2) * (16u", "(lane >> 1) * (16u"),
    ("weights", "const int b = 4 * (lane & 3) + i;\n", "const int b = 4 * (lane & 3) + i + 1;\n"),
    ("activations", "(uint32_t)(16 * (i >> 2) + (i & 3))", "(uint32_t)(4 * (i >> 2) + (i & 3))"),
    ("staged", "(chunk >> 2), nb) ? 0u", "(chunk >> 2) - 1, nb) ? 0u"),
    ("h", "2 * (n % kTileSlots)) * 16", "(n % kTileSlots)) * 16"),
    ("h", "(unit_start(u, nb) + b) * 1024", "(kUnit * u + b) * 1024"),
    ("tiles", "(slots < E ? slots : E) + slots / kTileSlots", "(slots < E ? slots : E) + slots / 16"),
])
def test_planted_mistakes_are_found(tmp_path, family, was, planted):
    with open(os.path.join(CSRC, "moe_offsets.hpp")) as f:
        text = f.read()
    assert text.count(was) == 1
    (tmp_path / "moe_offsets.hpp").write_text(text.replace(was, planted))
    assert _run(str(tmp_path), tmp_path)[0][family][1] > 0
