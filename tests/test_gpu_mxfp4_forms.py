"""Every form of the MXFP4 product's kernels, bit for bit: scales of 1/2, 1 and 2 make every product a
multiple of 1/16, and while a sum's magnitudes stay below 2^20 its partial sums have 24 bits, so that fp32
carries them exactly in any order and the one correct output is the exact sum rounded to bf16.
Each case names the form that it has to reach; ragged rows, widths and ends of K, and K beyond the
2048 elements that a group of scales covers."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host
from mx4_exact import guarded_u8, mxfp4_form, u8, values

pytestmark = pytest.mark.gpu

ROWS, SPLIT64, TILE64, TILE64X128, TILE128, TILE128X256, TILE256 = range(7)
CASES = [  # M, N, K, form
    (5, 257, 480, (ROWS, 16, 16, 8)), (16, 300, 1440, (ROWS, 16, 16, 8)),
    (2, 2106, 8192, (ROWS, 16, 16, 16)), (1, 301, 8224, (ROWS, 16, 16, 16)), (16, 100, 9024, (ROWS, 16, 16, 16)),
    (20, 301, 4128, (ROWS, 32, 16, 8)), (17, 4096, 512, (ROWS, 32, 16, 8)),
    (25, 4682, 768, (ROWS, 32, 32, 8)), (31, 8191, 800, (ROWS, 32, 32, 8)),
    (40, 301, 2016, (ROWS, 64, 16, 8)), (64, 1000, 4064, (ROWS, 64, 16, 8)),
    (100, 301, 2080, (SPLIT64, 64, 64, 3)), (41, 5001, 4192, (SPLIT64, 64, 64, 3)),
    (300, 1001, 992, (TILE64, 64, 64, 4)), (3344, 271, 2432, (TILE64, 64, 64, 4)),
    (1100, 2050, 992, (TILE64X128, 64, 128, 3)), (453, 4107, 2432, (TILE64X128, 64, 128, 3)),
    (1682, 2423, 2464, (TILE128, 128, 128, 2)), (2100, 2050, 4448, (TILE128, 128, 128, 2)),
    (1433, 1680, 1696, (TILE128, 128, 128, 4)), (401, 4673, 3136, (TILE128, 128, 128, 4)),
    (2837, 1488, 5760, (TILE128X256, 128, 256, 3)),
    (2777, 4501, 2432, (TILE256, 256, 256, 2)), (3333, 3999, 4448, (TILE256, 256, 256, 2)),
]
LINEAR = [  # M, N, K, form, one kernel
    (3, 301, 4096, (ROWS, 16, 16, 8), True), (16, 100, 1536, (ROWS, 16, 16, 8), True),
    (2, 2106, 8192, (ROWS, 16, 16, 16), True), (1, 333, 24576, (ROWS, 16, 16, 16), True),
    (2, 100, 16384, (ROWS, 16, 16, 16), False), (1, 8193, 1440, (SPLIT64, 64, 64, 3), False),
]
_ids = lambda c: "x".join(map(str, c[:3]))  # noqa: E731


def _operand(rows, K, seed):
    return guarded_u8(u8((rows, K // 2), seed)), guarded_u8(u8((rows, K // 32), seed + 1, 126, 129))


def _rounded(a, w):
    """The exact product rounded to bf16, and whether fp32 carries its sums."""
    a, w = values(*a), values(*w)
    assert float((a.abs() @ w.abs().T).max()) < 2.0**20
    return (a @ w.T).float().to(torch.bfloat16)



@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_product(case):
    M, N, K, form = case
    say("mxfp4 form", case)
    assert mxfp4_form(M, N, K)[0] == form
    a, w = _operand(M, K, 1), _operand(N, K, 3)
    out, ok = guarded((M, N), torch.bfloat16)
    nv.mxfp4_gemm(*a, *w, out=out)
    want = _rounded(a, w)
    differ = int((out != want).sum())
    assert differ == 0, f"{differ} of {M * N} outputs are not the rounded exact sum"
    assert ok()


@pytest.mark.parametrize("case", LINEAR, ids=_ids)
def test_linear(case):
    M, N, K, form, fused = case
    say("mxfp4 linear form", case)
    assert mxfp4_form(M, N, K) == (form, fused)
    # activations that are E2M1 values under their blocks' scales: quantization keeps them (each
    # block's largest is given as 6 or 4)
    a = _operand(M, K, 1)
    a[0].view(M, K // 32, 16)[:, :, 5] = 0x7E
    w = _operand(N, K, 3)
    x = nv.mxfp4_dequantize(*a)
    work = torch.empty(nv.mxfp4_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    out, ok = guarded((M, N), torch.bfloat16)
    nv.mxfp4_linear(x, *w, out=out, workspace=work)
    assert torch.equal(values(*nv.mxfp4_quantize(x)), values(*a))
    differ = int((out != _rounded(a, w)).sum())
    assert differ == 0, f"{differ} of {M * N} outputs are not the rounded exact sum"
    at = (M * K // 2 + 255) // 256 * 256
    p, s = nv.mxfp4_quantize(x)
    assert np.array_equal(to_host(work[: M * K // 2]), to_host(p).reshape(-1))
    assert np.array_equal(to_host(work[at: at + M * K // 32]), to_host(s).reshape(-1)) and ok()
