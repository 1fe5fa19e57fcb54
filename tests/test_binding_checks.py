"""The MXFP4 and mixture-of-experts binding's short argument checks, on tensors whose device number is that of the
host (-1): parameters pass them like plain tensors, and what is wrong still reaches the full check."""
import pytest
import torch

from nvfp4_block_scaled_02_amd import ops

U8 = torch.uint8


def _refuse(t, name, *_):
    raise ValueError(f"full check of {name}")


@pytest.fixture
def no_full_check(monkeypatch):
    monkeypatch.setattr(ops, "_need", _refuse)


def _tensors(*shape):
    t = torch.zeros(shape, dtype=U8)
    return t, torch.nn.Parameter(t, requires_grad=False)


def test_parameters_take_the_short_checks(no_full_check):
    for p in _tensors(4, 32):
        ops._want(p, "w", U8, 2, -1)
        for s in _tensors(4, 2):
            ops._want_pair(p, s, "w_", 2, -1)


def test_what_is_wrong_reaches_the_full_check(no_full_check):
    (p, q), (s, _) = _tensors(4, 32), _tensors(4, 2)
    for bad in (p.t(), p[0], p.int(), q.t(), None, [1]):
        with pytest.raises(ValueError, match="full check of w"):
            ops._want(bad, "w", U8, 2, -1)
        with pytest.raises(ValueError, match="full check of w_packed"):
            ops._want_pair(bad, s, "w_", 2, -1)
        with pytest.raises(ValueError, match="full check of w_scales"):
            ops._want_pair(p, bad, "w_", 2, -1)


def test_a_tensor_elsewhere_is_refused():
    with pytest.raises(ValueError, match="HIP device"):
        ops._want(torch.zeros(4, 32, dtype=U8), "w", U8, 2, 0)
