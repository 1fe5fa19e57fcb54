"""Argument checks of routing, the routed mixture of experts, low-rank adapters and the fused residual and
norm that need no GPU."""
import ctypes
import os

import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from nvfp4_block_scaled_02_amd import _lib as L

# Fake but aligned device addresses: validation never dereferences them.
P, Q, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0)
ODD8, ODD2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x20002)
INF, NAN = float("inf"), float("nan")


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


def test_moe_route(lib):
    #        logits bias T  E  k  scores groups top best renorm scale ids weights stream
    call = _caller(lib.nvfp4_moe_route, [P, P, 4, 64, 8, 1, 8, 4, 2, 1, 2.5, P, P, NULL])
    for k in (0, 11, 12):
        assert call({k: NULL}) == L.INVALID_VALUE
        assert call({k: ODD2}) == L.MISALIGNED
    assert call({1: ODD2}) == L.MISALIGNED
    for bad in ({5: 2}, {5: -1}, {8: 0}, {8: 3}, {9: 2}, {9: -1}, {10: NAN}, {10: INF}):
        assert call(bad) == L.INVALID_VALUE, bad
    for bad in ({2: -1}, {2: 2**21 + 1}, {3: 0}, {3: 513}, {3: 65}, {4: 0}, {4: 17}, {3: 4, 4: 5, 6: 1, 7: 1}, {6: 0}, {6: 65},
                {6: 7}, {6: 128, 3: 128}, {7: 0}, {7: 9}):
        assert call(bad) == L.INVALID_SHAPE, bad
    assert call({2: 0}) == L.SUCCESS and call({2: 0, 1: NULL}) == L.SUCCESS


def test_moe_routed(lib):
    need = lib.nvfp4_mxfp4_moe_workspace_bytes(4, 8, 64, 96, 2)
    #        x ids w w13 s13 w2 s2 T  E  H   I  k out work bytes stream
    call = _caller(lib.nvfp4_mxfp4_moe_routed, [P, Q, Q, P, Q, P, Q, 4, 8, 64, 96, 2, P, P, need, NULL])
    for k in (0, 1, 2, 3, 4, 5, 6, 12, 13):
        assert call({k: NULL}) == L.INVALID_VALUE
    for k in (0, 3, 5, 12, 13):
        assert call({k: ODD8}) == L.MISALIGNED
    for k in (1, 2, 4, 6):
        assert call({k: ODD2}) == L.MISALIGNED
    for bad in ({7: -1}, {7: 2**21 + 1}, {8: 0}, {8: 513}, {9: 48}, {10: 48}, {11: 0}, {11: 9}, {11: 17, 8: 32}):
        assert call(bad) == L.INVALID_SHAPE, bad
    assert call({14: need - 1}) == L.WORKSPACE
    assert call({7: 0}) == L.SUCCESS


def test_lora(lib):
    need = lib.nvfp4_lora_workspace_bytes(4, 100, 64, 40)
    assert need >= 4 * 40 * 4
    #        y x a b adapters scales T  N    K   R   L out work bytes stream
    call = _caller(lib.nvfp4_lora, [P, P, P, P, Q, Q, 4, 100, 64, 40, 3, P, P, need, NULL])
    for k in (0, 1, 2, 3, 4, 11, 12):
        assert call({k: NULL}) == L.INVALID_VALUE
    for k in (0, 1, 2, 3, 11, 12):
        assert call({k: ODD8}) == L.MISALIGNED
    for k in (4, 5):
        assert call({k: ODD2}) == L.MISALIGNED
    for bad in ({6: -1}, {6: 2**21 + 1}, {7: -1}, {7: 2**20 + 1}, {8: 0}, {8: 12}, {8: 2**20 + 8}, {9: 0}, {9: 12}, {9: 136},
                {10: -1}, {10: 2**31}):
        assert call(bad) == L.INVALID_SHAPE, bad
        if 10 not in bad:
            sizes = [4, 100, 64, 40]
            for k, v in bad.items():
                sizes[k - 6] = v
            assert lib.nvfp4_lora_workspace_bytes(*sizes) == 0
    assert call({13: need - 1}) == L.WORKSPACE
    assert lib.nvfp4_lora_workspace_bytes(1, 100, 64, 16) == 0  # few rows need none
    assert call({6: 0, 9: 16, 12: NULL, 13: 0}) == L.SUCCESS
    assert call({6: 0}) == L.SUCCESS and call({7: 0}) == L.SUCCESS and call({6: 0, 5: NULL, 10: 0}) == L.SUCCESS


def test_add_norm(lib):
    #        x y post gate c    w  b  sc sh rows M  H   G kind eps  h fmt gs gsdev out scales stream
    base = [P, P, P, P, 1.0, P, P, P, P, Q, 4, 64, 2, 0, 1e-6, P, 0, 0.0, NULL, P, NULL, NULL]
    call = _caller(lib.nvfp4_add_norm, base)
    for bad in ({0: NULL}, {19: NULL}, {15: NULL}, {1: NULL}, {1: NULL, 3: NULL}, {1: NULL, 2: NULL}, {13: 2}, {13: -1},
                {16: 5}, {16: -1}, {16: 2}, {14: 0.0}, {14: -1.0}, {14: NAN}, {14: INF}, {4: NAN}, {4: INF},
                {16: 1, 20: Q}, {16: 1, 20: Q, 17: -1.0}, {16: 1, 20: Q, 17: NAN}):
        assert call(bad) == L.INVALID_VALUE, bad
    for bad in ({10: -1}, {10: 2**31}, {11: 0}, {11: 12}, {11: 32776}, {12: 0}, {12: 3, 9: NULL}, {16: 2, 20: Q, 11: 48},
                {16: 3, 20: Q, 11: 48}, {16: 1, 20: Q, 17: 1.0, 11: 24}, {16: 4, 20: Q, 11: 24}):
        assert call(bad) == L.INVALID_SHAPE, bad
    for k in (0, 1, 2, 3, 5, 6, 7, 8, 15, 19):
        assert call({k: ODD8}) == L.MISALIGNED, k
    for bad in ({9: ODD2}, {16: 2, 20: ODD2}, {16: 1, 20: Q, 18: ODD2}):
        assert call(bad) == L.MISALIGNED, bad
    for good in ({}, {9: NULL}, {1: NULL, 2: NULL, 3: NULL, 15: NULL}, {16: 2, 20: Q}, {16: 1, 20: Q, 18: Q},
                 {16: 1, 20: Q, 17: 1.0}, {16: 4, 20: Q, 11: 16}, {11: 8}, {11: 32768}, {12: 7}):
        assert call({10: 0, **good}) == L.SUCCESS, good


def test_the_binding_refuses_what_is_not_on_a_device():
    f = torch.zeros(4, 64)
    h = f.to(torch.bfloat16)
    for call in (lambda: nv.moe_route(f, 2), lambda: nv.add_norm(h), lambda: nv.lora(h, h, h, h, f),
                 lambda: nv.mxfp4_moe_routed(h, f, f, f, f, f, f)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_workspace_grows_with_its_sizes(lib):
    for T in (1, 7, 64, 1000, 2**21):
        for K in (8, 512, 4104, 2**20):
            for R in (8, 24, 128):
                b = nv.lora_workspace_bytes(T, 64, K, R)
                assert b % 256 == 0 and (b >= 4 * T * R or (b == 0 and R <= 32))
