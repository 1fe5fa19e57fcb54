"""Argument checks of the MXFP4 and mixture-of-experts entry points that need no GPU."""
import ctypes
import os

import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from nvfp4_block_scaled_02_amd import _lib as L

# Fake but aligned device addresses: validation never dereferences them.
P, Q, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0)
ODD8, ODD2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x20002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from nvfp4_block_scaled_02_amd import build

        build.build()
    return L.load_library()


def _caller(fn, base):
    def call(changes):
        a = list(base)
        for k, v in changes.items():
            a[k] = v
        return fn(*a)

    return call


def test_quantize_and_dequantize(lib):
    for call in (_caller(lib.nvfp4_mxfp4_quantize, [P, 4, 64, P, Q, NULL]),):
        for k in (0, 3, 4):
            assert call({k: NULL}) == L.INVALID_VALUE
        for k in (0, 16, 48, -32):
            assert call({2: k}) == L.INVALID_SHAPE
        assert call({1: -1}) == L.INVALID_SHAPE
        assert call({1: 2**40, 2: 2**40}) == L.INVALID_SHAPE
        assert call({0: ODD8}) == L.MISALIGNED and call({3: ODD8}) == L.MISALIGNED
        assert call({4: ODD2}) == L.MISALIGNED
        assert call({1: 0}) == L.SUCCESS
    call = _caller(lib.nvfp4_mxfp4_dequantize, [P, Q, 4, 64, P, NULL])
    for k in (0, 1, 4):
        assert call({k: NULL}) == L.INVALID_VALUE
    assert call({3: 48}) == L.INVALID_SHAPE and call({2: -1}) == L.INVALID_SHAPE
    assert call({0: ODD8}) == L.MISALIGNED and call({1: ODD2}) == L.MISALIGNED and call({4: ODD8}) == L.MISALIGNED
    assert call({2: 0}) == L.SUCCESS


def test_gemm(lib):
    call = _caller(lib.nvfp4_mxfp4_gemm, [P, Q, P, Q, 8, 8, 64, P, NULL])
    for k in (0, 1, 2, 3, 7):
        assert call({k: NULL}) == L.INVALID_VALUE
    for k in (0, 16, 40, 2**22 + 32):
        assert call({6: k}) == L.INVALID_SHAPE
    for v in (-1, 2**31):
        assert call({4: v}) == L.INVALID_SHAPE and call({5: v}) == L.INVALID_SHAPE
    assert call({0: ODD8}) == L.MISALIGNED and call({2: ODD8}) == L.MISALIGNED and call({7: ODD8}) == L.MISALIGNED
    assert call({1: ODD2}) == L.MISALIGNED and call({3: ODD2}) == L.MISALIGNED
    assert call({4: 0}) == L.SUCCESS and call({5: 0}) == L.SUCCESS


def test_gemm_plan(lib):
    kind = ctypes.c_int(-1)
    call = _caller(lib.nvfp4_mxfp4_gemm_plan, [8, 8, 64, 0, ctypes.byref(kind)])
    assert call({4: None}) == L.INVALID_VALUE
    for k in (0, 16, 40, 2**22 + 32):
        assert call({2: k}) == L.INVALID_SHAPE
    for v in (-1, 2**31):
        assert call({0: v}) == L.INVALID_SHAPE and call({1: v}) == L.INVALID_SHAPE
    assert call({}) == L.SUCCESS and kind.value == 0  # rows
    assert nv.mxfp4_gemm_plan(8192, 8192, 8192) == "tile256"
    assert nv.mxfp4_gemm_plan(8192, 8192, 8192, 256) == nv.mxfp4_gemm_plan(8192, 8192, 8192, -1)


def test_gemm_plan_keeps_launches_below_two_to_the_32_threads(lib):
    """The widths at which the tile of least estimated time would have too many workgroups."""
    tiles = {"tile64": (64, 64), "tile64x128": (64, 128), "tile128": (128, 128), "tile128x256": (128, 256),
             "tile256": (256, 256)}
    top = 2**31 - 1
    for m, n in ((1, top), (top, 1), (64, top), (top, 64), (65, 2**30 + 1), (2**30 + 1, 65), (1, 2**30), (300, 2**29)):
        bm, bn = tiles[nv.mxfp4_gemm_plan(m, n, 32)]
        assert -(-m // bm) * -(-n // bn) * 256 < 2**32, (m, n)


def test_linear_and_its_workspace(lib):
    ws = lib.nvfp4_mxfp4_linear_workspace_bytes
    assert ws(8, 64) == 256 + 256 and ws(0, 64) == 0
    assert ws(1000, 4096) == 1000 * 2048 + (1000 * 128 + 255) // 256 * 256
    assert ws(8, 48) == 0 and ws(-1, 64) == 0
    call = _caller(lib.nvfp4_mxfp4_linear, [P, P, Q, 8, 8, 64, P, P, ws(8, 64), NULL])
    for k in (0, 1, 2, 6, 7):
        assert call({k: NULL}) == L.INVALID_VALUE
    assert call({8: ws(8, 64) - 1}) == L.WORKSPACE
    assert call({5: 48}) == L.INVALID_SHAPE and call({3: -1}) == L.INVALID_SHAPE
    assert call({0: ODD8}) == L.MISALIGNED and call({7: ODD8}) == L.MISALIGNED
    assert call({3: 0, 8: 0}) == L.SUCCESS


def test_router(lib):
    call = _caller(lib.nvfp4_moe_router, [P, P, 4, 8, 64, Q, NULL])
    for k in (0, 1, 5):
        assert call({k: NULL}) == L.INVALID_VALUE
    for ch in ({2: -1}, {2: 2**21 + 1}, {3: 0}, {3: 513}, {4: 0}, {4: 40}, {4: 2**20 + 32}):
        assert call(ch) == L.INVALID_SHAPE, ch
    assert call({0: ODD8}) == L.MISALIGNED and call({1: ODD8}) == L.MISALIGNED and call({5: ODD2}) == L.MISALIGNED
    assert call({2: 0}) == L.SUCCESS


def test_moe(lib):
    ws = lib.nvfp4_mxfp4_moe_workspace_bytes
    assert ws(4, 8, 64, 64, 2) > 4 * 2 * 64 * 2
    for bad in ((-1, 8, 64, 64, 2), (4, 0, 64, 64, 1), (4, 513, 64, 64, 2), (4, 8, 64, 48, 2), (4, 8, 48, 64, 2),
                (4, 8, 64, 64, 0), (4, 8, 64, 64, 9), (4, 32, 64, 64, 17)):
        assert ws(*bad) == 0, bad
    base = [P, Q, P, Q, P, Q, 4, 8, 64, 64, 2, 1, P, Q, Q, P, ws(4, 8, 64, 64, 2), NULL]
    call = _caller(lib.nvfp4_mxfp4_moe, base)
    for k in (0, 1, 2, 3, 4, 5, 12, 15):
        assert call({k: NULL}) == L.INVALID_VALUE
    assert call({11: 2}) == L.INVALID_VALUE
    for ch in ({6: -1}, {7: 0}, {7: 513}, {8: 48}, {8: 0}, {9: 48}, {9: -64}, {10: 0}, {10: 9}, {7: 32, 10: 17}):
        assert call(ch) == L.INVALID_SHAPE, ch
    for k in (0, 2, 4, 12, 15):
        assert call({k: ODD8}) == L.MISALIGNED
    for k in (1, 3, 5, 13, 14):
        assert call({k: ODD2}) == L.MISALIGNED
    assert call({16: ws(4, 8, 64, 64, 2) - 1}) == L.WORKSPACE
    # no tokens: success without a device, routing outputs optional
    assert call({6: 0, 13: NULL, 14: NULL}) == L.SUCCESS


def test_sizes_at_the_limits(lib):
    """Sizes and statuses of extreme shapes against exact integers: an overflow would show."""
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    values = [-(2**63), -1, 0, 1, 31, 32, 33, 64, 2**20, 2**20 + 32, 2**21, 2**21 + 1, 2**22, 2**22 + 32, 2**31 - 1,
              2**31, 2**32, 2**40, 2**62, 2**63 - 1, 2**63 - 32]
    kind = ctypes.c_int()
    for M in values:
        for K in values:
            ok = 0 <= M < 2**31 and 32 <= K <= 2**22 and K % 32 == 0
            assert lib.nvfp4_mxfp4_linear_workspace_bytes(M, K) == (up(M * K // 2) + up(M * K // 32) if ok else 0)
            for N in (-1, 0, 1, 2**31 - 1, 2**31):
                want = L.SUCCESS if ok and 0 <= N < 2**31 else L.INVALID_SHAPE
                assert lib.nvfp4_mxfp4_gemm_plan(M, N, K, 256, ctypes.byref(kind)) == want, (M, N, K)
    width = lambda v: 32 <= v <= 2**20 and v % 32 == 0  # noqa: E731
    for T in values:
        for E in (0, 1, 512, 513, 2**40):
            for H in values[3:]:
                for I in (32, 2**20, 2**20 + 32):
                    got = lib.nvfp4_mxfp4_moe_workspace_bytes(T, E, H, I, 1)
                    assert (got > 0) == (0 < T <= 2**21 and 1 <= E <= 512 and width(H) and width(I)), (T, E, H, I)
                    if got:  # at least every chunk's h, and below what a sum past 2^63 would wrap to
                        assert -(-T // 64) * 32 * I <= got < 2**62


def test_no_device_is_reported(lib, gpu_available):
    if gpu_available:
        pytest.skip("a GPU is present")
    assert lib.nvfp4_mxfp4_quantize(P, 4, 64, P, Q, NULL) == L.UNSUPPORTED_DEVICE
    assert lib.nvfp4_mxfp4_dequantize(P, Q, 4, 64, P, NULL) == L.UNSUPPORTED_DEVICE
    assert lib.nvfp4_mxfp4_gemm(P, Q, P, Q, 8, 8, 64, P, NULL) == L.UNSUPPORTED_DEVICE
    assert lib.nvfp4_mxfp4_linear(P, P, Q, 8, 8, 64, P, P, 512, NULL) == L.UNSUPPORTED_DEVICE
    assert lib.nvfp4_moe_router(P, P, 4, 8, 64, Q, NULL) == L.UNSUPPORTED_DEVICE
    assert lib.nvfp4_mxfp4_moe(P, Q, P, Q, P, Q, 4, 8, 64, 64, 2, 1, P, NULL, NULL, P, 1 << 20, NULL) == \
        L.UNSUPPORTED_DEVICE


def test_binding_refuses_host_tensors_and_types():
    bf, u8 = torch.bfloat16, torch.uint8
    x, p, s = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8)
    for call in (lambda: nv.mxfp4_quantize(x), lambda: nv.mxfp4_dequantize(p, s),
                 lambda: nv.mxfp4_gemm(p, s, p, s), lambda: nv.mxfp4_linear(x, p, s),
                 lambda: nv.moe_router(x, x)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    for call in (lambda: nv.mxfp4_quantize(x.float()), lambda: nv.mxfp4_dequantize(x, s),
                 lambda: nv.mxfp4_gemm(x, s, p, s), lambda: nv.moe_router(x.half(), x)):
        with pytest.raises(TypeError):
            call()
