"""MXFP4 and mixture-of-experts calls with an empty side: refused as the same call with one row is, and doing what
the call still has to do."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import to_host

pytestmark = pytest.mark.gpu

BF, U8 = torch.bfloat16, torch.uint8


def _new(*shape, dtype=U8):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _moe(T, E, H, I, k, **kw):
    return nv.mxfp4_moe(_new(T, H, dtype=BF), _new(T, E, dtype=torch.float32), _new(E, 2 * I, H // 2),
                        _new(E, 2 * I, H // 32), _new(E, H, I // 2), _new(E, H, I // 32), k, **kw)


@pytest.mark.parametrize("T", [0, 1])
def test_layer(T):
    for k in (0, -1, 5, 17):
        with pytest.raises(nv.NVFP4Error):
            _moe(T, 4, 64, 32, k)
    with pytest.raises(nv.NVFP4Error):
        _moe(T, 32, 64, 32, 17)
    for E, H, I in ((513, 64, 32), (0, 64, 32), (4, 64, 0)):
        with pytest.raises(nv.NVFP4Error):
            _moe(T, E, H, I, 1)
    out, ids, weights = _moe(T, 4, 64, 32, 2, return_routing=True)
    assert out.shape == (T, 64) and ids.shape == weights.shape == (T, 2)


@pytest.mark.parametrize("T", [0, 1])
def test_router(T):
    for E, H in ((0, 64), (513, 64), (4, 48), (4, 0)):
        with pytest.raises(nv.NVFP4Error):
            nv.moe_router(_new(T, H, dtype=BF), _new(E, H, dtype=BF))
    assert nv.moe_router(_new(T, 64, dtype=BF), _new(4, 64, dtype=BF)).shape == (T, 4)


@pytest.mark.parametrize("M", [0, 1])
def test_product_and_linear(M):
    for N in (0, 3):
        for K in (0, 16):
            with pytest.raises(nv.NVFP4Error):
                nv.mxfp4_gemm(_new(M, K // 2), _new(M, K // 32), _new(N, K // 2), _new(N, K // 32))
            with pytest.raises(nv.NVFP4Error):
                nv.mxfp4_linear(_new(M, K, dtype=BF), _new(N, K // 2), _new(N, K // 32))
        with pytest.raises(nv.NVFP4Error):   # a workspace too small by a byte, misaligned
            nv.mxfp4_linear(_new(1, 64, dtype=BF), _new(N, 32), _new(N, 2), workspace=_new(511))
        with pytest.raises(nv.NVFP4Error):
            nv.mxfp4_linear(_new(M, 64, dtype=BF), _new(N, 32), _new(N, 2), workspace=_new(1024)[8:])
        assert nv.mxfp4_linear(_new(M, 64, dtype=BF), _new(N, 32), _new(N, 2)).shape == (M, N)


@pytest.mark.parametrize("M", [0, 1])
def test_format(M):
    with pytest.raises((ValueError, nv.NVFP4Error)):
        nv.mxfp4_quantize(_new(M, 0, dtype=BF))
    with pytest.raises((ValueError, nv.NVFP4Error)):
        nv.mxfp4_dequantize(_new(M, 0), _new(M, 0))
    p, s = nv.mxfp4_quantize(_new(M, 64, dtype=BF))
    assert p.shape == (M, 32) and s.shape == (M, 2) and nv.mxfp4_dequantize(p, s).shape == (M, 64)


def test_a_linear_without_outputs_still_leaves_the_quantized_activations():
    x = torch.randn((5, 96), device="cuda").to(BF)
    work = torch.full((nv.mxfp4_linear_workspace_bytes(5, 96),), 0xEE, dtype=U8, device="cuda")
    assert nv.mxfp4_linear(x, _new(0, 48), _new(0, 3), workspace=work).shape == (5, 0)
    p, s = nv.mxfp4_quantize(x)
    assert np.array_equal(to_host(work[:240]), to_host(p).reshape(-1))
    assert np.array_equal(to_host(work[256:271]), to_host(s).reshape(-1))
