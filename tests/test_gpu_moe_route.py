"""Routing to experts on the GPU against 64 bits: ids exactly, weights to one rounding."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _logits(T, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, E), device="cuda", generator=g) * 1.5


def _check(l, k, **how):
    T, E = l.shape
    say("route", T, E, k, {n: (v if n != "bias" else v is not None) for n, v in how.items()})
    ids, ok_i = guarded((T, k), torch.int32)
    weights, ok_w = guarded((T, k), torch.float32)
    assert nv.moe_route(l, k, ids=ids, weights=weights, **how)[0] is ids
    bias = how.pop("bias", None)
    wid, wwt = BO.route(to_host(l), k, bias=None if bias is None else to_host(bias), **how)
    bad = np.flatnonzero((to_host(ids) != wid).any(1))
    assert bad.size == 0, f"rows {bad[:5]}: {to_host(ids)[bad[:5]].tolist()} for {wid[bad[:5]].tolist()}"
    got = to_host(weights).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(wwt))
    fine = ~np.isnan(wwt)
    assert (np.abs(got - wwt)[fine] <= BO.route_tol(wwt)[fine]).all()
    assert ok_i() and ok_w()
    return ids, weights


SHAPES = [  # T, E, top_k, groups, top_groups
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (2, 8, 8, 1, 1), (3, 60, 4, 1, 1), (5, 60, 5, 6, 2), (7, 160, 6, 8, 3), (64, 64, 6, 64, 7),
    (65, 65, 3, 5, 4), (33, 128, 16, 4, 1), (4, 512, 16, 64, 9), (9, 512, 1, 2, 1), (130, 200, 7, 10, 10), (17, 12, 12, 3, 2),
    (6, 63, 2, 63, 5), (3, 200, 16, 4, 2)]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_route(shape, scores):
    T, E, k, groups, top = shape
    l = _logits(T, E, sum(shape))
    bias = _logits(1, E, 3)[0] * 0.1
    for b in (None, bias):
        for best in (1, 2):
            for renormalize in (False, True):
                _check(l, k, scores=scores, bias=b, groups=groups, top_groups=top, group_best=best,
                       renormalize=renormalize, scale=2.5 if b is None else 1.0)


@pytest.mark.parametrize("E,groups,top", [(12, 1, 1), (12, 4, 2), (96, 3, 2), (320, 32, 3), (64, 4, 2), (160, 8, 3), (512, 16, 5), (48, 2, 1)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_masked_and_unordered(E, groups, top, scores):
    k, low = 4, torch.finfo(torch.float32).min
    l = _logits(18, E, E)
    l[0] = -INF                      # padding
    l[1, 1:] = -INF                  # one expert
    l[2] = low                       # the type's lowest value is a value like any other
    l[3], l[3, 7] = low, 0.0
    l[4, : E // 2] = -INF            # whole groups that are not there
    l[5, ::2] = -INF
    l[6] *= 1e30
    l[7] = 3.4e38
    l[8, 0], l[8, 1:] = 88.0, -88.0
    l[9] = 0.0                       # ties
    l[10] = -900.0 - torch.arange(E, device="cuda")  # scores that 64 bits have no room for
    l[11], l[11, 3] = 0.0, -0.0
    l[12] = 100.0 + torch.arange(E, device="cuda") % 5  # sigmoids that are all 1
    l[13, 2:] = -INF
    l[14] = 60.0 + 30.0 * torch.arange(E, device="cuda") / E   # the same, in rising order
    l[15] = -800.0 - torch.arange(E, device="cuda").flip(0)    # far from the first one
    l[15, 0] = 0.0
    l[16] = -45.0 - torch.arange(E, device="cuda") % 7
    l[17] = torch.arange(E, device="cuda") % 3 - 30.0
    bias = torch.linspace(0.2, -0.2, E, device="cuda")
    off = bias.clone()
    off[::3] = -INF                  # experts that are switched off
    for renormalize in (True, False):
        for best in (1, 2):
            for b in (None, bias, off):
                _check(l, k, scores=scores, bias=b, groups=groups, top_groups=top, group_best=best, renormalize=renormalize)


def test_nan_and_infinite_logits():
    E, k = 40, 3
    l = _logits(4, E, 1)
    l[0, 17] = NAN
    l[1, 5], l[1, 9] = NAN, NAN
    l[2] = NAN
    l[3, 11] = INF
    for renormalize in (True, False):
        _check(l, k, scores="sigmoid", renormalize=renormalize)
        _check(l, k, scores="sigmoid", renormalize=renormalize, bias=torch.zeros(E, device="cuda"))
        _check(l, k, scores="sigmoid", renormalize=renormalize, groups=8, top_groups=3, group_best=2)
        # under softmax the sum over all experts is NaN
        ids, w = nv.moe_route(l, k, renormalize=renormalize)
        assert to_host(ids)[:, 0].tolist() == [17, 5, 0, 11] and np.isnan(to_host(w)).all()


def test_bias_that_ties_keys_and_next_neighbours():
    """Keys that differ in their last bits of 64, and not at all."""
    E = 64
    l = torch.zeros((3, E), device="cuda")
    l[1, 10] = 1e-7                  # next to the others
    l[2] = torch.arange(E, device="cuda") * 1e-6
    bias = torch.zeros(E, device="cuda")
    bias[40] = 2.0**-30
    for scores in ("softmax", "sigmoid"):
        ids, _ = _check(l, 4, scores=scores, bias=bias)
        assert to_host(ids)[0].tolist() == [40, 0, 1, 2]


@pytest.mark.parametrize("T", [0, 4099, 70000])
def test_many_tokens(T):
    E, k = 96, 6
    l = _logits(T, E, 7)
    bias = _logits(1, E, 8)[0] * 0.05
    how = dict(scores="sigmoid", bias=bias, groups=8, top_groups=3, group_best=2, scale=2.5)
    ids, w = nv.moe_route(l, k, **how)
    assert ids.shape == (T, k) and w.shape == (T, k)
    if T:
        at = torch.randint(0, T, (60,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        few, fw = _check(l[at].contiguous(), k, **how)
        assert torch.equal(ids[at], few) and torch.equal(w[at], fw)  # a token's result is its own


def test_agrees_with_the_layer_that_routes_for_itself():
    l = _logits(50, 72, 2)
    for renormalize in (True, False):
        ids, w = nv.moe_route(l, 6, renormalize=renormalize)
        from oracle import mxfp4_oracle as M4
        wid, wwt = M4.route(to_host(l), 6, renormalize)
        assert np.array_equal(to_host(ids), wid) and np.allclose(to_host(w), wwt, rtol=2.0**-23, atol=0)


def test_refusals():
    l = _logits(4, 8, 1)
    for bad in (dict(scores="relu"), dict(bias=torch.zeros(7, device="cuda")), dict(bias=torch.zeros(8)),
                dict(ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            nv.moe_route(l, 2, **bad)
    for bad in (dict(groups=3), dict(groups=0), dict(top_groups=2), dict(group_best=3), dict(scale=NAN)):
        with pytest.raises(nv.NVFP4Error):
            nv.moe_route(l, 2, **bad)
    for k in (0, 9, -1):
        with pytest.raises(nv.NVFP4Error):
            nv.moe_route(l, k)
    with pytest.raises(TypeError):
        nv.moe_route(l.half(), 2)
    with pytest.raises(ValueError):
        nv.moe_route(l.t(), 2)


def _next(x, n):
    """x moved by n steps of fp32."""
    return float((np.float32(x).view(np.int32) + n).view(np.float32)) if x > 0 else -_next(-x, -n)


@pytest.mark.parametrize("E,groups,top", [(16, 1, 1), (60, 1, 1), (64, 4, 2), (160, 8, 3), (256, 8, 4), (512, 16, 5), (96, 12, 4)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_neighbours_a_few_steps_apart(E, groups, top, scores):
    """Rows whose first, second, last and next choices lie one to a few hundred steps of fp32 apart, in either order
    of index, alone and in runs: where 32-bit keys do not tell."""
    k = 6
    rows = []
    r = np.random.default_rng(E)
    for trial in range(64):
        l = r.standard_normal(E).astype(np.float32)
        order = np.argsort(-l)
        for at in ((0,), (k - 2,), (k - 1,), (k,), (0, k - 1), (k - 1, k), (k - 1, k, k + 1), tuple(range(k + 2)))[trial % 8]:
            if at + 1 < E:
                step = int(r.choice([0, 1, 2, 7, 30, 300])) * int(r.choice([-1, 1]))
                l[order[at + 1]] = _next(float(l[order[at]]), step) if l[order[at]] != 0 else 0.0
        rows.append(l)
    l = torch.from_numpy(np.stack(rows)).cuda()
    bias = torch.from_numpy((0.05 * r.standard_normal(E)).astype(np.float32)).cuda()
    flat = torch.full((E,), 0.125, device="cuda")  # every key moved alike: neighbours stay neighbours
    for b in (None, flat, bias):
        for best in (1, 2):
            _check(l, k, scores=scores, bias=b, groups=groups, top_groups=top, group_best=best, renormalize=best == 1)
