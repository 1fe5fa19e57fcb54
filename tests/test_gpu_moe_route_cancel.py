"""Groups whose two largest keys cancel: one large bias for and one against, so that the keys' own roundings in 32 bits are more than
what tells the sums apart; ids exactly, weights to one rounding, against 64 bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


def _inputs(T, E, groups, b, scores, seed):
    """In each group one expert with a bias of +b, the others of -b. The sum of its two largest scores is 0.9 and a few roundings
    of b in fp32 more or less, other in each group; 2^-24 to 2^-12 at least."""
    r = np.random.default_rng(seed)
    size = E // groups
    for_ = r.integers(0, size, groups)
    step = np.minimum(max(b * 2.0**-24, 2.0**-24) * 2.0 ** r.uniform(0, 4, (T, 1)), 0.2 / groups)  # (scores stay in (0, 1))
    total = 0.9 + step * r.permuted(np.tile(np.arange(groups) - groups // 2, (T, 1)), axis=1) * r.uniform(0.5, 1.5, (T, groups))
    second = r.uniform(0.3, 0.6, (T, groups))
    s = r.uniform(0.01, 0.2, (T, groups, size))
    for g in range(groups):
        s[:, g, for_[g]] = total[:, g] - second[:, g]
        s[:, g, (for_[g] + 1 + r.integers(0, size - 1)) % size] = second[:, g]
    l = np.log(s) if scores == "softmax" else np.log(s / (1.0 - s))
    bias = np.full((groups, size), -b)
    bias[np.arange(groups), for_] = b
    assert np.isfinite(l).all()
    return l.reshape(T, E).astype(np.float32), bias.reshape(E).astype(np.float32)


def _check(l, k, bias, **how):
    ids, weights = nv.moe_route(torch.from_numpy(l).cuda(), k, bias=torch.from_numpy(bias).cuda(), **how)
    want, weight = BO.route(l, k, bias=bias, **how)
    bad = np.flatnonzero((to_host(ids) != want).any(1))
    assert bad.size == 0, f"{bad.size} rows, {bad[:3]}: {to_host(ids)[bad[:3]].tolist()} for {want[bad[:3]].tolist()}"
    assert (np.abs(to_host(weights).astype(np.float64) - weight) <= BO.route_tol(weight)).all()


@pytest.mark.parametrize("b", [0.25, 1.0, 4.0, 16.0, 1000.0, 1e6])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 4), (256, 8, 3), (64, 4, 2), (128, 16, 7)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_sums_that_cancel(E, groups, top, b, scores):
    T = 500 if b >= 16 else 200
    say("cancel", T, E, groups, b, scores)
    l, bias = _inputs(T, E, groups, b, scores, E + int(b))
    for renormalize in (True, False):
        _check(l[:: 1 if renormalize else 7], 6, bias, scores=scores, groups=groups, top_groups=top, group_best=2, renormalize=renormalize)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_some_groups_cancel_beside_others_that_do_not(scores):
    """Sums near each other of keys large and small."""
    T, E, groups = 600, 128, 8
    say("mixed", scores)
    for b in (2.0, 64.0, 3e4):
        l, bias = _inputs(T, E, groups, b, scores, 5)
        bias = bias.reshape(groups, -1)
        bias[::2] = np.where(bias[::2] > 0, 0.0, bias[::2] * 1e-6)  # (its own size is of no account beside the others' sums)
        _check(l, 6, bias.reshape(-1), scores=scores, groups=groups, top_groups=4, group_best=2)
