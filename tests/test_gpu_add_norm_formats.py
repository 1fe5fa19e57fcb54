"""The norm's quantized results byte for byte the quantizers', in all formats: many rows, and NaN and infinities in rows and in
single columns (NVFP4 has no NaN: of such an element the code is left open, and that alone)."""
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say

pytestmark = pytest.mark.gpu

FORMATS = {"nvfp4": lambda n, gs: nv.quantize(n, gs), "mxfp4": lambda n, gs: nv.mxfp4_quantize(n),
           "mxfp8": lambda n, gs: nv.mxfp8_quantize(n), "fp8r": lambda n, gs: nv.fp8r_quantize(n)}


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _same(fmt, *args, **how):
    gs = 0.01 if fmt == "nvfp4" else None
    h, n = nv.add_norm(*args, **how)
    want = FORMATS[fmt](n, gs)
    h2, got = nv.add_norm(*args, quantize=fmt, global_scale=gs, **how)
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))
    assert torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8))
    known = torch.ones_like(n, dtype=torch.bool)
    if fmt == "nvfp4":  # has no NaN: such an element's code is not defined, all others are
        known = ~torch.isnan(n)
        got, want = (torch.stack((q[0] & 15, q[0] >> 4), dim=-1).flatten(1) for q in (got, want))
        clean = FORMATS[fmt](torch.nan_to_num(n, nan=0.0, posinf=float("inf"), neginf=float("-inf")), gs)
        clean = torch.stack((clean[0] & 15, clean[0] >> 4), dim=-1).flatten(1)
        assert torch.equal(want[known], clean[known])  # as if it were a zero
    else:
        got, want = got[0], want[0]
        known = known if got.shape == n.shape else torch.ones_like(got, dtype=torch.bool)
    assert torch.equal(got[known], want[known])
    return n


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [64, 1056, 2080, 4128, 16416])
def test_bad_values(H, kind, fmt):
    say("bad values", fmt, kind, H)
    M, nan, inf = 9, float("nan"), float("inf")
    x, y, w, b = _bf16((M, H), 1, 3.0), _bf16((M, H), 2), _bf16((H,), 3), _bf16((H,), 4)
    x[2, 5], x[3, H - 1], y[4, 40], x[5, 3], x[5, 4] = nan, inf, -inf, inf, -inf
    x[6], y[6] = 0.0, 0.0
    n = _same(fmt, x, y, weight=w, kind=kind)
    assert torch.isnan(n[2]).all() and torch.isfinite(n[[0, 1, 6, 7, 8]].float()).all()
    for i, v in enumerate((nan, inf, -inf)):  # of one column in every row
        b2 = b.clone()
        b2[33 + i] = v
        n = _same(fmt, x, y, weight=w, bias=b2, kind=kind)
        assert not torch.isfinite(n[:, 33 + i].float()).any()
        w2 = w.clone()
        w2[H - 1 - i] = v
        _same(fmt, x, y, weight=w2, kind=kind)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_rows(fmt):
    M, H = 3000, 1056
    say("many rows", fmt)
    x, y, w = _bf16((M, H), 1, 3.0), _bf16((M, H), 2), _bf16((H,), 3)
    x[5, 40], x[6, 41] = float("nan"), float("inf")
    _same(fmt, x, y, weight=w)
