"""Operand reads of the MXFP4 product's kernels, modelled on the CPU: ``tests/native/
mx4_bounds_check.cpp`` evaluates the offset functions that the kernels call
(``csrc/mx4_offsets.hpp``) over ragged shapes and checks that none leaves its operand or row."""
import os
import subprocess

import pytest

import nvfp4_block_scaled_02_amd as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def report(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("mx4") / "mx4_bounds_check")
    cmd = ["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17",
           "-I", os.path.join(ROOT, "nvfp4_block_scaled_02_amd", "csrc"), "-I", os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "native", "mx4_bounds_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=600)


@pytest.mark.parametrize("family", ["tiles", "rows"])
def test_no_read_leaves_its_operand(report, family):
    line = [l for l in report.stdout.splitlines() if l.startswith(family + " reads ")]
    assert line, report.stdout + report.stderr
    reads, bad = line[0].split(" reads ")[1].split(" violations ")
    assert int(reads) > 10000 and int(bad) == 0, line[0] + "\n" + report.stderr


def test_plan_keeps_the_kernels_within_their_lengths():
    """The kernel that splits K needs K > 1024; every kernel is reached."""
    seen = set()
    for K in (32, 480, 512, 992, 1024, 1056, 2048, 4096, 8192):
        for M in (1, 16, 17, 33, 40, 64, 100, 333, 1024, 2048, 4096, 8192):
            for N in (1, 64, 1000, 4096, 8192, 14336):
                kind = nv.mxfp4_gemm_plan(M, N, K)
                seen.add(kind)
                if kind == "split64":
                    assert K > 1024, (M, N, K)
                if kind == "rows":
                    assert M <= 64
    assert seen == {"rows", "split64", "tile64", "tile64x128", "tile128", "tile128x256", "tile256"}
    assert nv.mxfp4_gemm_plan(1, 64, 1 << 20) == "split64"   # scales of 16 rows of K exceed the LDS
    assert nv.mxfp4_gemm_plan(300, 4096, 4096, 64) != nv.mxfp4_gemm_plan(300, 4096, 4096)
