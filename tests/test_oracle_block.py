"""The 64-bit references of routing, low-rank adapters and the fused residual and norm, pinned to worked
examples and closed forms (CPU)."""
import numpy as np
import pytest

from oracle import block_oracle as BO

INF, NAN = float("inf"), float("nan")


def test_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]], np.float32))
    ids, w = BO.route(l, 2, renormalize=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]], atol=1e-7)
    ids, w = BO.route(l, 2, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]], atol=1e-6)
    ids, w = BO.route(l, 2, bias=np.array([0.4, 0, 0, 0], np.float32), renormalize=False)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[0.125, 0.5]], atol=1e-7)  # the bias chooses, the score weighs
    ids, w = BO.route(np.zeros((1, 4), np.float32), 3, scores="sigmoid", renormalize=False)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.5, 0.5, 0.5]]


def test_route_groups_by_hand():
    l = np.array([[5.0, 0.0, 3.0, 2.9, 4.0, -9.0]], np.float32)  # groups (0,1) (2,3) (4,5)
    assert BO.route(l, 2, groups=3, top_groups=1)[0].tolist() == [[0, 1]]
    ids, _ = BO.route(l, 4, scores="sigmoid", groups=3, top_groups=1, group_best=2)
    assert ids.tolist() == [[2, 3, -1, -1]]  # .953 + .948 against .993 + .5, .982 + 0
    ids, w = BO.route(l, 4, groups=3, top_groups=2)
    assert ids.tolist() == [[0, 4, 1, 5]] and np.isclose(w.sum(), 1.0)


def test_route_masked():
    l = np.array([[-INF, -INF, -INF], [-INF, 1.0, -INF], [NAN, 0.0, 1.0], [-800.0, -801.0, -INF]], np.float32)
    ids, w = BO.route(l, 2, scores="sigmoid")
    assert ids.tolist() == [[-1, -1], [1, -1], [0, 2], [0, 1]]
    assert w[0].tolist() == [0.0, 0.0] and w[1].tolist() == [1.0, 0.0] and np.isnan(w[2]).all()
    assert np.allclose(w[3], [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))])
    assert BO.route(l, 2, bias=np.array([0, -INF, 0], np.float32), scores="sigmoid")[0][1].tolist() == [-1, -1]


def test_lora_by_hand():
    y, x = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([[1.0, -1.0], [2.0, 0.5]])
    a, b = np.array([[[2.0, 1.0]]]), np.array([[[3.0], [-1.0]]])
    out, tol = BO.lora(y, x, a, b, np.array([-1, 0]), np.array([0.5], np.float32))
    assert out.tolist() == [[1.0, 2.0], [3.0 + 0.5 * 4.5 * 3, 4.0 - 0.5 * 4.5]]
    assert (tol[0] < 1e-30).all() and (tol[1] >= BO.B * np.abs(out[1])).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_closed_forms(kind):
    v = np.array([[3.0, -3.0, 3.0, -3.0], [0.0, 0.0, 0.0, 0.0]])
    n, tol = BO.normed(v, kind, 1e-12, weight=np.array([1.0, 2.0, 1.0, 1.0]), bias=np.ones(4))
    assert np.allclose(n[0], [2.0, -1.0, 2.0, 0.0]) and np.allclose(n[1], 1.0)
    n, _ = BO.normed(v + 5.0, kind, 1e-12)
    want = v if kind == "layer" else v + 5.0
    assert np.allclose(n[0], want[0] / np.sqrt((want[0] ** 2).mean()))
    h, _ = BO.residual(v, 2 * v + 1, kind, 1e-12, gate=np.full((2, 1), 0.5), c=4.0)
    assert np.allclose(h, v + 4.0 * 0.5 * (2 * v + 1))


def test_tolerances_tell_a_mistake():
    r = np.random.default_rng(0)
    h, w = r.standard_normal((3, 64)), r.standard_normal(64)
    n, tol = BO.normed(h, "rms", 1e-6, weight=w)
    wrong, _ = BO.normed(h, "layer", 1e-6, weight=w)
    assert (np.abs(wrong - n) > tol).any()
    wrong, _ = BO.normed(h, "rms", 1e-6, weight=np.roll(w, 1))
    assert (np.abs(wrong - n) > tol).any()
    y, x = r.standard_normal((4, 8)), r.standard_normal((4, 32))
    a, b = r.standard_normal((2, 8, 32)), r.standard_normal((2, 8, 8))
    out, tol = BO.lora(y, x, a, b, np.array([0, 1, -1, 0]))
    for adapters in ([1, 1, -1, 0], [0, 1, 0, 0], [0, -1, -1, 0]):
        assert (np.abs(BO.lora(y, x, a, b, np.array(adapters))[0] - out) > tol).any()
