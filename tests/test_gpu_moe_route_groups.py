"""Groups of experts ranked by the sum of their two largest keys, where 32 bits do not hold the sum or do not tell two sums apart;
ids exactly, weights to one rounding, against 64 bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
INF, LOW = float("inf"), float(np.finfo(np.float32).min)


def _check(l, k, bias, **how):
    say("route", *l.shape, k, how)
    ids, weights = nv.moe_route(torch.from_numpy(l).cuda(), k, bias=torch.from_numpy(bias).cuda(), **how)
    want, weight = BO.route(l, k, bias=bias, **how)
    bad = np.flatnonzero((to_host(ids) != want).any(1))
    assert bad.size == 0, f"{bad.size} rows, {bad[:3]}: {to_host(ids)[bad[:3]].tolist()} for {want[bad[:3]].tolist()}"
    assert (np.abs(to_host(weights).astype(np.float64) - weight) <= BO.route_tol(weight)).all()
    return want


@pytest.mark.parametrize("second", [(-INF, LOW, LOW), (-3e38, -2e38, -3e38)], ids=["lowest", "below"])
def test_sums_below_the_range_of_32_bits(second):
    """Group 0 has two experts, its own best ones; the others' two best keys add up to less than fp32 holds."""
    l = np.zeros((3, 64), np.float32)
    l[:, 1], l[:, 32] = 1.0, 0.5
    bias = np.repeat(np.array((0.0,) + second), 16) * np.where(np.isinf(second[0]), 1.0, 1.0 - 0.02 * (np.arange(64) % 16))
    bias[2:16] = -INF
    want = _check(l, 4, bias.astype(np.float32), scores="sigmoid", groups=4, top_groups=2, group_best=2)
    assert (want[:, :2] == [1, 0]).all() and (want[:, 2:] // 16 == 2).all()


@pytest.mark.parametrize("E,groups,top", [(32, 16, 5), (64, 4, 2), (64, 8, 4), (256, 8, 3), (128, 2, 1), (60, 10, 3)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_biases_at_the_ends_of_the_range(E, groups, top, scores):
    """Experts switched off by -inf, by the lowest value and by other large ones, in any mix; and preferred by as much."""
    r = np.random.default_rng(E + groups)
    for values in ((0.0, -INF, LOW), (0.0, LOW), (-INF, LOW, -2e38, -1.8e38, -1.6e38), (0.1, -INF, LOW, -LOW, 3e38, -3e38, 2e38, 1e30),
                   (-1e9, 0.0, -INF), (LOW,)):
        bias = r.choice(np.array(values, np.float32), E)
        l = (1.5 * r.standard_normal((40, E))).astype(np.float32)
        l[::4, : E // 2] = -INF
        l[1::4, ::2] = -INF
        for best in (1, 2):
            _check(l, 4, bias, scores=scores, groups=groups, top_groups=top, group_best=best, renormalize=best == 1)
