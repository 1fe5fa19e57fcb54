"""Accesses and launches of the low-rank adapters' kernels, modelled on the CPU: ``tests/native/lora_bounds_check.cpp``
evaluates the functions that the kernels call (``csrc/lora_offsets.hpp``)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_02_amd", "csrc")
FAMILIES = ("staged", "columns", "neighbours", "forms")


def _run(folder, first=CSRC):
    exe = os.path.join(folder, "lora_bounds_check")
    cmd = ["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17", "-I", str(first), "-I", CSRC,
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "lora_bounds_check.cpp"), "-o", exe]
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
        assert n > 100 and v == 0, (family, n, v, err)


@pytest.mark.parametrize("family, was, planted", [
    ("staged", "unit * kC + chunk < chunks ? 0u", "unit * kC + chunk <= chunks ? 0u"),
    ("staged", "k * (64 / kC) + lane / kC", "k * (64 / kC) + lane / 16"),
    ("staged", "^ (row & 15)", "^ (row & 31)"),
    ("columns", "16 * (r >> 2) + 4 * i", "16 * (r >> 2) + 3 * i"),
    ("neighbours", "(xcd < more ? xcd : more)", "xcd"),
    ("forms", "lora_clamp((work + 511) / 512, 1, 16)", "lora_clamp((work + 511) / 512, 1, 1)"),
])
def test_planted_mistakes_are_found(tmp_path, family, was, planted):
    with open(os.path.join(CSRC, "lora_offsets.hpp")) as f:
        text = f.read()
    assert text.count(was) == 1, text.count(was)
    (tmp_path / "lora_offsets.hpp").write_text(text.replace(was, planted))
    assert _run(str(tmp_path), tmp_path)[0][family][1] > 0
