"""The sizes of the GPU tests that compare bit for bit reach every form of the MXFP4 product's and the
mixture-of-experts layer's kernels that some size takes (host only)."""
import random

import test_gpu_moe_exact as moe
import test_gpu_mxfp4_forms as product
from mx4_exact import moe_form, mxfp4_form
from nvfp4_block_scaled_02_amd import ops


def _log(rng, lo, hi):
    return int(lo * (hi / lo) ** rng.random())


def test_product():
    rng, seen = random.Random(1), set()
    for _ in range(100000):
        seen.add(mxfp4_form(_log(rng, 1, 9000), _log(rng, 1, 20000), 32 * _log(rng, 1, 400))[0])
    for M, N, K, form in product.CASES:
        assert mxfp4_form(M, N, K)[0] == form, (M, N, K)
    assert {c[3] for c in product.CASES} == seen
    fused = {(c[3], c[4]) for c in product.LINEAR}
    for M, N, K, form, one in product.LINEAR:
        assert mxfp4_form(M, N, K) == (form, one), (M, N, K)
    assert {f for f, one in fused if one} == {(0, 16, 16, 8), (0, 16, 16, 16)}
    assert len(seen) == 12 and ops.MXFP4_KERNELS.keys() == {f[0] for f in seen}


def test_layer():
    rng, seen = random.Random(2), set()
    for _ in range(100000):
        T, E = _log(rng, 1, 400), _log(rng, 1, 513)
        seen.add(moe_form(T, E, rng.randint(1, min(E, 16)), 32 * _log(rng, 1, 200), 32 * _log(rng, 1, 400)))
    for case in moe.CASES + moe.WIDEST + moe.LARGE:
        assert moe_form(*case[:5]) == case[5], case
    assert {c[5] for c in moe.CASES} == seen
    # the forms of many tokens at more than 64, which are planned in several chunks
    assert {c[5] for c in moe.CASES if c[0] > 64} == {f for f in seen if f[0] == 2}


def test_the_layers_form_goes_by_units():
    """Widths of the same number of units of 512 elements take the same form of the first product."""
    for T, E, k, I in ((64, 32, 4, 1440), (64, 128, 8, 1024), (40, 64, 6, 1408), (64, 8, 8, 2048), (4, 16, 2, 2048)):
        for units in range(1, 14):
            assert len({moe_form(T, E, k, H, I) for H in range(512 * units - 480, 512 * units + 1, 32)}) == 1, (T, E, units)


def test_linear_in_one_kernel_is_what_the_header_says():
    rng = random.Random(3)
    for _ in range(20000):
        M, N, K = _log(rng, 1, 40), _log(rng, 1, 20000), 32 * _log(rng, 1, 1000)
        assert mxfp4_form(M, N, K)[1] == (M <= 16 and M * K <= 24576 and N <= 8192), (M, N, K)
    for M, N, K in ((1, 8192, 24576), (1, 8193, 32), (16, 8192, 1536), (16, 8192, 1568), (17, 64, 32), (1, 1, 24608)):
        assert mxfp4_form(M, N, K)[1] == (M <= 16 and M * K <= 24576 and N <= 8192), (M, N, K)
