"""Low-rank adapters on the GPU against 64 bits, within the bound counted in oracle/block_oracle.py."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _f64(t):
    return to_host(t.float()).astype(np.float64)


def _inputs(T, N, K, R, L, seed):
    y, x = _bf16((T, N), seed), _bf16((T, K), seed + 1)
    a, b = _bf16((L, R, K), seed + 2, K**-0.5), _bf16((L, N, R), seed + 3, R**-0.5)
    scales = torch.rand((L,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) + 0.25
    return y, x, a, b, scales


def _run(y, x, a, b, adapters, scales=None, out=None):
    """The call, its workspace and output between canaries, the workspace full of NaN."""
    T, N, K, R = *y.shape, x.shape[1], a.shape[1]
    work, ok_w = guarded((nv.lora_workspace_bytes(T, N, K, R),), torch.uint8, fill=0xFF)
    res, ok = (out, lambda: True) if out is not None else guarded((T, N), torch.bfloat16)
    nv.lora(y, x, a, b, adapters, scales=scales, out=res, workspace=work)
    assert ok() and ok_w(), "wrote outside its buffers"
    return res


def _check(y, x, a, b, adapters, scales, label):
    L = a.shape[0]
    say("lora", label, *y.shape, tuple(a.shape))
    before = y.clone()
    got = _run(y, x, a, b, adapters, scales)
    assert torch.equal(y.view(torch.int16), before.view(torch.int16))
    ad = to_host(adapters)
    ref, tol = BO.lora(_f64(y), _f64(x), _f64(a), _f64(b), np.where((ad >= 0) & (ad < L), ad, -1),
                       None if scales is None else to_host(scales))
    err = np.abs(_f64(got) - ref)
    assert (err <= tol).all(), f"{label}: worst {np.max(err / tol):.3g} of the bound"
    none = torch.from_numpy((ad < 0) | (ad >= L)).cuda()
    assert torch.equal(got[none].view(torch.int16), y[none].view(torch.int16))
    again = y.clone()
    assert torch.equal(_run(again, x, a, b, adapters, scales, out=again).view(torch.int16), got.view(torch.int16))
    return got


def _adapters(T, L, how, seed):
    r = np.random.default_rng(seed)
    if how == "each":      # a decode batch
        ad = r.integers(-1, L, T)
    elif how == "runs":    # prompts of different lengths
        ends = np.sort(r.integers(0, T + 1, 5))
        ad = np.repeat(r.integers(-1, L, 6), np.diff(np.concatenate(([0], ends, [T]))))
    else:                  # all the same
        ad = np.full(T, L // 2)
    return torch.from_numpy(ad.astype(np.int32)).cuda()


CASES = [  # T, N, K, R, L
    (1, 1, 8, 8, 1), (1, 256, 512, 16, 3), (1, 4096, 4096, 16, 2), (2, 17, 40, 24, 2), (5, 1001, 2560, 32, 6), (15, 64, 264, 40, 4),
    (16, 65, 256, 48, 2), (17, 63, 72, 56, 20), (33, 130, 1032, 64, 3), (48, 333, 288, 72, 32), (64, 256, 512, 96, 2),
    (100, 96, 96, 104, 100), (255, 24, 136, 120, 3), (257, 100, 520, 128, 9), (300, 1024, 64, 8, 5), (1023, 72, 200, 16, 4),
    (2000, 520, 256, 64, 7), (4100, 33, 48, 32, 2),
    # many rows: all ranks of two tiles at once, several tiles per workgroup of the second product, v shared or not
    (4100, 64, 136, 40, 3), (5000, 24, 4104, 72, 4), (4128, 200, 264, 128, 5), (4100, 2056, 72, 64, 5), (20000, 520, 40, 16, 6),
    (9000, 4104, 64, 128, 3), (6001, 1023, 128, 96, 2), (3000, 4096, 520, 56, 4)]


@pytest.mark.parametrize("how", ["each", "runs", "same"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_lora(case, how):
    T, N, K, R, L = case
    y, x, a, b, scales = _inputs(*case, sum(case))
    _check(y, x, a, b, _adapters(T, L, how, sum(case)), scales if how != "runs" else None, how)


@pytest.mark.parametrize("T", [3, 16, 70, 600])
def test_rows_without_an_adapter(T):
    N, K, R, L = 130, 96, 16, 3
    y, x, a, b, scales = _inputs(T, N, K, R, L, 1)
    y[0, 0] = float("nan")
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(_run(y, x, a, b, none, scales).view(torch.int16), y.view(torch.int16))
    y, x, a, b, scales = _inputs(T, N, K, R, L, 1)
    ad = none.clone()
    ad[0], ad[T // 2], ad[T - 1] = L, 2**31 - 1, -(2**31)  # past either end
    assert torch.equal(_run(y, x, a, b, ad, scales).view(torch.int16), y.view(torch.int16))
    ad[1] = 2
    _check(y, x, a, b, ad, scales, "one row")
    empty = a[:0], b[:0], scales[:0]
    assert torch.equal(_run(y, x, empty[0], empty[1], torch.zeros_like(ad), empty[2]).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("T", [4, 40, 400, 5000])
def test_a_row_depends_on_its_own_adapter_and_activations_alone(T):
    """NaN and infinities in other adapters' weights, scales and other rows leave a row as it is."""
    N, K, R, L = (200, 328, 24, 4) if T < 5000 else (1200, 328, 72, 4)
    y, x, a, b, scales = _inputs(T, N, K, R, L, 5)
    ad = _adapters(T, 3, "each", 2)
    ad[0], ad[1] = 0, 3
    clean = _run(y, x, a, b, torch.where(ad == 3, -1, ad), scales)
    bad = [t.clone() for t in (x, a, b, scales)]
    bad[0][1], bad[1][3], bad[2][3, ::2], bad[2][3, 1::2], bad[3][3] = float("nan"), float("inf"), float("nan"), -float("inf"), 3e38
    got = _run(y, *bad[:3], ad, bad[3])
    rows = ad != 3
    assert torch.equal(got[rows].view(torch.int16), clean[rows].view(torch.int16))
    assert not torch.isfinite(got[~rows].float()).all()


def test_infinite_and_large_products():
    """A x that overflows fp32 gives infinities and NaN as the formula does; at 2^100 it is an ordinary number."""
    y, x, a, b, _ = _inputs(20, 64, 64, 8, 1, 9)
    ad = torch.zeros(20, dtype=torch.int32, device="cuda")
    big = (x.float() * 2.0**100).to(torch.bfloat16)
    got = _check((y.float() * 2.0**100).to(torch.bfloat16), big, a, b, ad, None, "2^100")
    assert torch.isfinite(got.float()).all()
    x = torch.full_like(x, 3e38)
    a, b = torch.full_like(a, 2.0), torch.full_like(b, 1.0)
    assert (_run(y, x, a, b, ad) == float("inf")).all()


def test_a_result_is_the_same_every_time():
    for T, L in ((7, 3), (200, 16), (3000, 5)):
        y, x, a, b, scales = _inputs(T, 333, 520, 32, L, T)
        ad = _adapters(T, L, "each", 1)
        first = _run(y, x, a, b, ad, scales)
        for _ in range(3):
            assert torch.equal(_run(y, x, a, b, ad, scales).view(torch.int16), first.view(torch.int16))


def test_far_offsets():
    """Adapters and outputs past 2^31 elements: the last adapter of many, the last rows of a wide output."""
    K, N, R, L = 8, 65536, 128, 300  # b: 2.5e9 elements
    say("far adapters")
    y, x = _bf16((20, N), 1), _bf16((20, K), 2)
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda")
    a[L - 1], b[L - 1] = _bf16((R, K), 3), _bf16((N, R), 4, 0.1)
    ad = torch.full((20,), L - 1, dtype=torch.int32, device="cuda")
    got = _run(y, x, a, b, ad)
    ref, tol = BO.lora(_f64(y), _f64(x), _f64(a[L - 1:]), _f64(b[L - 1:]), np.zeros(20, np.int64))
    assert (np.abs(_f64(got) - ref) <= tol).all()
    del b, y, got
    say("far rows")
    T, N = 2**16 + 3, 2**15 + 7  # 2.1e9 elements of y
    y, x = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"), _bf16((T, K), 2)
    a, b = _bf16((1, 8, K), 3), _bf16((1, N, 8), 4)
    ad = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ad[T - 2] = ad[T - 40] = 0
    got = nv.lora(y, x, a, b, ad)
    at = [T - 40, T - 2, T - 1]
    ref, tol = BO.lora(np.zeros((3, N)), _f64(x[at]), _f64(a), _f64(b), np.array([0, 0, -1]))
    assert (np.abs(_f64(got[at]) - ref) <= tol).all()
    got[at] = 0
    assert not got.any()


def test_empty():
    y, x, a, b, s = _inputs(4, 32, 64, 8, 2, 1)
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert nv.lora(y[:0], x[:0], a, b, ad[:0]).shape == (0, 32)
    assert nv.lora(y[:, :0].contiguous(), x, a, b[:, :0].contiguous(), ad).shape == (4, 0)


def test_refusals():
    y, x, a, b, s = _inputs(4, 32, 64, 8, 2, 1)
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((y, x[:3].contiguous(), a, b, ad), (y, x, a, b[:1].contiguous(), ad), (y, x, a, b[:, :31].contiguous(), ad),
                (y, x, a, b, ad[:3]), (y, x, a, b, ad.cpu()), (y.t(), x, a, b, ad), (y, x, a[0], b, ad),
                (y, x, a, b, ad, s[:1]), (y, x, a, b, ad, s, y[:2])):
        with pytest.raises(ValueError):
            nv.lora(*bad)
    for bad in ((y.float(), x, a, b, ad), (y, x, a.half(), b, ad), (y, x, a, b, ad.long()), (y, x, a, b, ad, s.double())):
        with pytest.raises(TypeError):
            nv.lora(*bad)
    with pytest.raises(nv.NVFP4Error):
        nv.lora(y, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ad)
    y, x, a, b, s = _inputs(4, 32, 64, 40, 2, 1)
    with pytest.raises(nv.NVFP4Error):
        nv.lora(y, x, a, b, ad, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
