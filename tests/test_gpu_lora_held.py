"""Between its two products the adapters' A x is held in 32 bits: sums of B's that cancel all but its last bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host

pytestmark = pytest.mark.gpu

CASES = [  # T, N, K, R: one launch, one or two fragments of ranks per workgroup, many rows; v shared by the waves or not
    (1, 40, 64, 8), (5, 300, 4096, 16), (16, 64, 200, 24), (33, 130, 1032, 32), (70, 33, 24, 40), (300, 520, 256, 48),
    (1000, 256, 264, 64), (2000, 72, 136, 72), (3000, 64, 72, 96), (4100, 520, 96, 64), (4200, 200, 520, 104), (6001, 1023, 40, 128),
    (20000, 264, 64, 16), (9000, 2056, 40, 120)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_last_bits_of_the_first_product(case):
    _last_bits(case, 0, 0)


@pytest.mark.parametrize("case", [(1, 40, 64, 8), (16, 64, 200, 24), (300, 520, 256, 48), (4100, 520, 96, 64)], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("x_power, a_power", [(-50, -59), (-60, -20), (60, 60)])
def test_last_bits_of_small_and_large_products(case, x_power, a_power):
    """The same where v is 2^-109, whose last part is below the least normal bf16, and 2^120."""
    _last_bits(case, x_power, a_power)


def _last_bits(case, x_power, a_power):
    """x of a row holds 1.0 to 1.98, 2^-8 to 2^-7 and 2^-16 to 2^-15 in 8 bits each. Even ranks add all three, 24 bits, and
    odd ones the first two, both exactly in any order; an output column takes p (v_even - v_odd), the third value alone.
    Its six products (three parts each) and y = 0 are added within 2^-24 of at most 2 p each: 8 2^-24 2 p = 2^-20 p. v held
    in 16 bits would be off by up to 2^-16 p."""
    T, N, K, R = case
    say("lora held", *case)
    r = np.random.default_rng(sum(case))
    where = (0, K // 2, K - 1)
    x, third = np.zeros((T, K), np.float32), (r.integers(128, 256, T) * 2.0**-23).astype(np.float32)
    x[:, where[0]] = r.integers(128, 254, T) / 128.0
    x[:, where[1]] = r.integers(128, 256, T) * 2.0**-15
    x[:, where[2]] = third
    a, b = np.zeros((2, R, K), np.float32), np.zeros((2, N, R), np.float32)
    a[:, :, where[0]] = a[:, :, where[1]] = 1.0
    a[:, ::2, where[2]] = 1.0
    n = np.arange(N)
    p = (2.0 ** (n % 5)).astype(np.float32)
    pair = 2 * (n % (R // 2))
    b[0, n, pair], b[0, n, pair + 1] = p, -p
    b[1] = -b[0]
    # exact powers: v = A x takes 2^(x + a), B takes it back, as far as bf16 goes
    x, a, b = (np.ldexp(t, e).astype(np.float32) for t, e in ((x, x_power), (a, a_power), (b, -(x_power + a_power))))
    adapters = r.integers(0, 2, T).astype(np.int32)
    x, a, b = (torch.from_numpy(t).cuda().to(torch.bfloat16) for t in (x, a, b))
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    scales = torch.tensor([2.0, 0.5], device="cuda")
    got = to_host(nv.lora(y, x, a, b, torch.from_numpy(adapters).cuda(), scales).float()).astype(np.float64)
    factor = np.where(adapters == 0, 2.0, -0.5)[:, None] * p[None, :]
    assert (np.abs(got - third[:, None] * factor) <= 2.0**-20 * np.abs(factor)).all()
