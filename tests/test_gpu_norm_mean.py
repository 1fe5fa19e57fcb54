"""The layer norm's mean: rows far from zero, against 64 bits, within the roundings of what is left after the mean."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
WIDTHS = [24, 504, 520, 1000, 1032, 1160, 2056, 3000, 4104, 6152, 8192, 16392, 32760]


def _f64(t):
    return to_host(t.float()).astype(np.float64)


@pytest.mark.parametrize("H", WIDTHS)
def test_constant_rows_are_zero(H):
    """Sums of up to 2^15 equal values of 8 bits are exact in fp32, and so is their quotient by H: nothing is left."""
    say("constant rows", H)
    values = torch.tensor([1000.0, 30080.0, -77.5, 3.0, 1e15, -1e-3, 255.0], device="cuda")
    x = values.to(torch.bfloat16)[:, None].repeat(1, H)
    bias = torch.linspace(-1, 1, H, device="cuda").to(torch.bfloat16)
    _, n = nv.add_norm(x, kind="layer", bias=bias)
    assert torch.equal(n, bias[None, :].expand_as(n))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    h, _ = nv.add_norm(torch.zeros_like(x), x, post_weight=w, kind="layer")
    assert not h.any()


@pytest.mark.parametrize("H", WIDTHS)
def test_rows_far_from_zero(H):
    """One value a step from the others, several steps, and a spread far below the mean."""
    say("rows far from zero", H)
    g = torch.Generator(device="cuda").manual_seed(H)
    noise = torch.randn((6, H), device="cuda", generator=g)
    x = torch.tensor([1000.0, 30080.0, -77.0, 5e8, 1000.0, -3e4], device="cuda")[:, None].repeat(1, H)
    x[0, H // 3] += 4.0              # a step of bf16 at 1000
    x[1, -1] -= 128.0
    x[2] += 0.5 * (noise[2] > 2)
    x[3] += 2.0**21 * noise[3].round()
    x[4] += 4.0 * noise[4].round()
    x[5] += 100.0 * noise[5]
    x = x.to(torch.bfloat16)
    _, n = nv.add_norm(x, kind="layer", eps=1e-5)
    want, tol = BO.normed(_f64(x), "layer", 1e-5)
    err = np.abs(_f64(n) - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the bound"
    assert (tol <= 0.004 * np.abs(want) + 3e-4).all()  # the bound says something: little above the output's own rounding
