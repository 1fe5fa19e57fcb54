"""The order in which the low-rank adapters' second product takes the parts of its operand, on the CPU:
``tests/native/lora_parts_check.cpp`` evaluates the functions that the kernels call (``csrc/lora_offsets.hpp``)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_02_amd", "csrc")


def _run(folder, first=CSRC):
    exe = os.path.join(folder, "lora_parts_check")
    cmd = ["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17", "-I", str(first), "-I", CSRC,
           "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "native", "lora_parts_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    _, _, n, _, v = r.stdout.split()
    return int(n), int(v), r.stderr


def test_every_part_meets_its_weights(tmp_path):
    n, v, err = _run(str(tmp_path))
    assert n > 1000 and v == 0, err


@pytest.mark.parametrize("was, planted", [("4 * k + q < R / 4 ?", "4 * k + q <= R / 4 ?"), ("lower < R / 8 ? R / 4 +", "lower < R / 8 ? R / 8 +"),
                                          ("return R % 32 == 0;", "return R % 16 == 0;")])
def test_planted_mistakes_are_found(tmp_path, was, planted):
    with open(os.path.join(CSRC, "lora_offsets.hpp")) as f:
        text = f.read()
    assert text.count(was) == 1, text.count(was)
    (tmp_path / "lora_offsets.hpp").write_text(text.replace(was, planted))
    assert _run(str(tmp_path), tmp_path)[1] > 0
