"""The mixture-of-experts layer with its routing given: bit for bit the layer that routes for itself, and routings
that it would not make (indices that are no expert's, the same expert twice, rows without any)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host
from oracle import mxfp4_oracle as M4
from test_gpu_moe import CASES, _bf16, _experts

pytestmark = pytest.mark.gpu


def _routed(x, ids, weights, dev):
    T, H = x.shape
    E, I = dev[0].shape[0], dev[0].shape[1] // 2
    out, ok = guarded((T, H), torch.bfloat16)
    work, ok_w = guarded((nv.mxfp4_moe_workspace_bytes(T, E, H, I, ids.shape[1]),), torch.uint8, fill=0xFF)
    before = ids.clone(), weights.clone()
    nv.mxfp4_moe_routed(x, ids, weights, *dev, out=out, workspace=work)
    assert ok() and ok_w()
    assert torch.equal(ids, before[0]) and torch.equal(weights.view(torch.int32), before[1].view(torch.int32))
    return out


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_same_routing_same_bits(case):
    T, E, k, H, I = case
    say("routed", *case)
    x, (_, dev) = _bf16((T, H), 1), _experts(E, H, I, 2)
    l = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    l[T // 2, 1:] = -float("inf")
    want, ids, weights = nv.mxfp4_moe(x, l, *dev, k, return_routing=True)
    got = _routed(x, ids, weights, dev)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T", [1, 2, 4, 5, 16, 17, 64, 65, 130])
def test_odd_routings(T):
    """The same expert in every slot, in some, indices past either end, and rows with nothing."""
    E, k, H, I = 12, 6, 160, 96
    say("odd routings", T)
    x, (w, dev) = _bf16((T, H), 4), _experts(E, H, I, 5)
    r = np.random.default_rng(T)
    ids = r.integers(0, E, (T, k)).astype(np.int32)  # repeats at random
    weights = r.standard_normal((T, k)).astype(np.float32)
    ids[0] = 3
    if T > 1:
        ids[1] = [-1, E, 2**31 - 1, -(2**31), E + 5, -7]
    if T > 3:
        ids[2], ids[3] = [5, -1, 5, E, 0, 5], [-1, -1, -1, -1, -1, 11]
        weights[3, :5] = np.nan  # of no expert
    got = to_host(_routed(x, torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), dev).float())
    mine = np.where((ids >= 0) & (ids < E), ids, -1)
    ref, tol = M4.moe_ref(to_host(x.float()).astype(np.float64), mine, np.where(mine < 0, 0.0, weights).astype(np.float64),
                          M4.dequantize(*w[:2]), M4.dequantize(*w[2:]))
    assert (np.abs(got - ref) <= tol + 1e-37).all()
    if T > 1:
        assert not got[1].any()


def test_every_token_at_one_expert_with_every_slot():
    """64 tokens whose 16 slots are all one expert's: 1024 of them, where an expert has room for 64."""
    T, E, k, H, I = 64, 16, 16, 96, 1088
    say("one expert")
    x, (w, dev) = _bf16((T, H), 1), _experts(E, H, I, 2)
    ids = torch.full((T, k), 7, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), 1.0 / 16, device="cuda")
    alone, one = torch.full((T, k), -1, dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    alone[:, 0], one[:, 0] = 7, 1.0
    a, b = _routed(x, ids, weights, dev), _routed(x, alone, one, dev)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_refusals():
    T, E, k, H, I = 4, 8, 2, 64, 96
    x, (_, dev) = _bf16((T, H), 1), _experts(E, H, I, 2)
    ids, weights = torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    with pytest.raises(ValueError):
        nv.mxfp4_moe_routed(x, ids[:3].contiguous(), weights, *dev)
    with pytest.raises(ValueError):
        nv.mxfp4_moe_routed(x, ids, weights[:, :1].contiguous(), *dev)
    with pytest.raises(TypeError):
        nv.mxfp4_moe_routed(x, ids.long(), weights, *dev)
    with pytest.raises(ValueError):
        nv.mxfp4_moe_routed(x, ids, weights.cpu(), *dev)
    with pytest.raises(nv.NVFP4Error):
        nv.mxfp4_moe_routed(x, ids, weights, *dev, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        nv.mxfp4_moe_routed(x, ids[:, :0].contiguous(), weights[:, :0].contiguous(), *dev)
    assert nv.mxfp4_moe_routed(x[:0], ids[:0], weights[:0], *dev).shape == (0, H)
