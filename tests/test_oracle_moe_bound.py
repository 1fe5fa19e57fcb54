"""The mixture-of-experts oracle tells results apart: a float32 computation is within its bound and
correctly rounded nearly everywhere; one with h rounded to bf16 is not correctly rounded, an empty one, another
expert's and one with a missing block of K are out of the bound. (The bound's sums are worst cases, n 2^-24
of the magnitudes: from some hundred elements of H on they hide a rounding of h, the share of
outputs that differ from the rounded exact value does not.)"""
import numpy as np
import pytest

from oracle import mxfp4_oracle as M4
from oracle.nvfp4_oracle import bf16_bits_to_f32
from workloads import to_bf16_bits

H_ERROR = 2.0**-16  # h in two bf16 parts, the first cut, the second rounded


def _bf16(a):
    return bf16_bits_to_f32(to_bf16_bits(a.astype(np.float32))).astype(np.float64)


def _parts(a):
    """h as two bf16 parts: the upper half of its float32, and the rest rounded."""
    hi = (a.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    return hi.astype(np.float64) + _bf16(a - hi)


def _layer(x, ids, weights, w13, w2, h_as=lambda a: a.astype(np.float64)):
    """The layer in float32 sums, one bf16 rounding of the output."""
    I = w2.shape[2]
    out = np.zeros(x.shape, dtype=np.float32)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            gu = w13[e].astype(np.float32) @ x[t].astype(np.float32)
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            y = (w2[e] @ h_as(h)).astype(np.float32)
            out[t] += np.float32(weights[t, j]) * y
    return _bf16(out)


@pytest.mark.parametrize("size", [(3, 4, 2, 64, 96), (8, 4, 4, 96, 64), (4, 3, 1, 512, 128)], ids=str)
def test_bound_tells_results_apart(size):
    T, E, k, H, I = size
    rng = np.random.default_rng(sum(size))
    x = _bf16(rng.standard_normal((T, H)))
    w13 = M4.dequantize(rng.integers(0, 256, (E, 2 * I, H // 2), dtype=np.uint8),
                        rng.integers(121, 124, (E, 2 * I, H // 32)).astype(np.uint8))
    w2 = M4.dequantize(rng.integers(0, 256, (E, H, I // 2), dtype=np.uint8),
                       rng.integers(121, 124, (E, H, I // 32)).astype(np.uint8))
    ids, weights = M4.route(rng.standard_normal((T, E)).astype(np.float32), k, True)
    ref, tol = M4.moe_ref(x, ids, weights, w13, w2, H_ERROR)
    inside = lambda out: np.abs(out - ref) <= tol  # noqa: E731
    assert inside(_layer(x, ids, weights, w13, w2)).all()
    assert inside(_layer(x, ids, weights, w13, w2, _parts)).all()
    # h rounded to bf16: within the wider bound, and outside this one at many outputs
    coarse = _layer(x, ids, weights, w13, w2, _bf16)
    assert (np.abs(coarse - ref) <= M4.moe_ref(x, ids, weights, w13, w2)[1]).all()
    differ = lambda out: (out != _bf16(ref)).mean()  # noqa: E731
    assert differ(coarse) > 0.1
    assert differ(_layer(x, ids, weights, w13, w2)) < 0.02 and differ(_layer(x, ids, weights, w13, w2, _parts)) < 0.02
    assert (~inside(np.zeros_like(ref))).mean() > 0.95
    assert (~inside(_layer(x, (ids + 1) % E, weights, w13, w2))).mean() > 0.9
    short = x.copy()
    short[:, 32:64] = 0.0   # a block of K left out
    assert (~inside(_layer(short, ids, weights, w13, w2))).mean() > 0.9


def test_two_parts_hold_a_value_to_sixteen_bits():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(200000) * np.exp(rng.uniform(-60, 60, 200000))).astype(np.float32)
    v[:3] = [np.float32(3.4028235e38), -np.float32(3.3961776e38), np.float32(1.0) + np.float32(2.0**-16)]
    assert (np.abs(_parts(v) - v) <= H_ERROR * np.abs(v)).all()
