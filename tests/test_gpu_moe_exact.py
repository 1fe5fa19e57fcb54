"""The mixture-of-experts layer bit for bit, in every form of its kernels, at its limits and past 2^32 bytes.

Activations are a power of two at 2^n places of a token's row and 0 elsewhere, gate weights are all 4: the
gate is a power of two of at least 128, of which silu is the same number in fp32 (exp(-128) is below its
range), and exact in any order of the sum only if every place is taken once. The up rows have random codes under scales of 1/2, 1
and 2, so that h is a whole number of few bits. Logits are 0 at top_k chosen experts, a power of two of them,
and -200 elsewhere, so that their weights are 1 / top_k. While magnitudes stay below 2^24 steps, all sums are
exact in fp32 in any order, and the one correct output is the exact value rounded to bf16."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say
from mx4_exact import guarded_u8, moe_form, u8, values

pytestmark = pytest.mark.gpu

INLINE, PLAN, ROUTE = range(3)
CASES = [  # T, E, top_k, H, I, (who routes, staged, few, shares)
    (1, 1, 1, 32, 32, (INLINE, 0, 0, 0)), (4, 32, 4, 544, 96, (INLINE, 0, 0, 0)), (3, 8, 2, 2080, 1440, (INLINE, 0, 0, 0)),
    (4, 64, 16, 96, 256, (INLINE, 1, 1, 0)), (3, 64, 8, 2080, 1056, (INLINE, 1, 1, 0)),
    (5, 4, 4, 64, 96, (PLAN, 0, 0, 1)), (12, 8, 2, 544, 96, (PLAN, 0, 0, 1)), (16, 4, 4, 2080, 544, (PLAN, 0, 0, 1)),
    (16, 64, 8, 544, 544, (PLAN, 1, 1, 1)), (9, 64, 8, 2592, 1440, (PLAN, 1, 1, 1)),
    (20, 8, 2, 544, 96, (ROUTE, 0, 0, 1)), (64, 4, 4, 1056, 544, (ROUTE, 0, 0, 1)), (130, 4, 2, 544, 96, (ROUTE, 0, 0, 1)),
    (64, 128, 8, 544, 160, (ROUTE, 1, 1, 1)), (65, 32, 4, 544, 1088, (ROUTE, 1, 1, 1)), (130, 32, 4, 544, 1088, (ROUTE, 1, 1, 1)),
    (300, 64, 8, 1056, 544, (ROUTE, 1, 1, 1)),
    (64, 8, 8, 544, 2080, (ROUTE, 1, 0, 1)), (65, 4, 2, 544, 8704, (ROUTE, 1, 0, 1)), (130, 4, 2, 544, 8704, (ROUTE, 1, 0, 1)),
    (64, 32, 8, 4128, 1056, (ROUTE, 1, 0, 1)), (200, 16, 4, 4128, 1056, (ROUTE, 1, 0, 1)),
]
WIDEST = [(3, 1, 1, 2**20, 32, (INLINE, 0, 0, 0)), (6, 1, 1, 2**20, 32, (PLAN, 0, 0, 1)),
          (70, 1, 1, 2**20, 32, (ROUTE, 0, 0, 1)), (2, 1, 1, 32, 2**20, (INLINE, 1, 1, 0)),
          (6, 1, 1, 32, 2**20, (PLAN, 1, 1, 1)), (70, 1, 1, 32, 2**20, (ROUTE, 1, 0, 1))]
LARGE = [(2, 512, 2, 8192, 1024, (INLINE, 0, 0, 0)), (6, 512, 2, 8192, 1024, (PLAN, 0, 0, 1)),
         (20, 512, 2, 8192, 1024, (ROUTE, 1, 0, 1)), (70, 512, 2, 8192, 1024, (ROUTE, 1, 0, 1))]
_ids = lambda c: "x".join(map(str, c[:5]))  # noqa: E731


def _weights(E, H, I, k, ones, seed):
    """Of W2 all blocks have codes, or one in so many that the sums stay exact: the mean magnitude of
    a code is 2.6, of an element of h 3.1 sqrt(ones), each in quarters."""
    sparse = 1
    while k * I * 2.6 * 3.1 * np.sqrt(ones) * 16 / sparse > 2**23:
        sparse *= 2
    w13, s13 = u8((E, 2 * I, H // 2), seed), u8((E, 2 * I, H // 32), seed + 1, 126, 129)
    w13[:, :I], s13[:, :I] = 0x66, 127
    w2, s2 = u8((E, H, I // 2), seed + 2), u8((E, H, I // 32), seed + 3, 126, 129)
    if sparse > 1:
        keep = u8((E, H, I // 32, 1), seed + 4) < 256 // sparse
        keep[:, :, [0, -1]] = True
        w2 = (w2.view(E, H, I // 32, 16) * keep).view(E, H, I // 2)
    return w13, s13, w2, s2


def _activations(T, H, ones, seed):
    """``ones`` equal powers of two a token at the ends of the row, around the ends of units of 512, and anywhere."""
    rng = np.random.default_rng(seed)
    x = np.zeros((T, H), dtype=np.float32)
    for t in range(T):
        edges = np.unique(np.clip(np.concatenate([[0, H - 1], 512 * rng.integers(0, H // 512 + 1, ones // 8) +
                                                  rng.integers(-1, 1, ones // 8)]), 0, H - 1))
        rest = rng.permutation(np.setdiff1d(np.arange(H), edges))
        at = np.concatenate([edges, rest])[:ones]
        x[t, at] = 2.0 ** (max(0, 5 - int(np.log2(ones))) + t % 3)
    return torch.from_numpy(x).to("cuda").to(torch.bfloat16)


def _exact(x, chosen, w, k, shift=0):
    """The layer in float64, the largest sum of magnitudes of an output in steps (u and W2 are quarters of a
    token's power of two and of one; the gate and the weights 1 / top_k are powers of two), and the largest u
    in steps."""
    T, H = x.shape
    I = w[2].shape[2] * 2
    out, most = torch.zeros((T, H), dtype=torch.float64, device="cuda"), torch.zeros((T, H), dtype=torch.float64, device="cuda")
    xd, u_most = x.double(), 0.0
    power = xd.amax(1, keepdim=True)
    for e in np.unique(chosen.cpu().numpy()).tolist():
        if e < 0:
            continue
        t = (chosen == e).any(1).nonzero()[:, 0]
        f = (e + shift) % w[0].shape[0]
        g = 4.0 * xd[t].sum(1, keepdim=True)
        up = torch.cat([xd[t] @ values(p, s).T for p, s in zip(w[0][f, I:].split(4096), w[1][f, I:].split(4096))], dim=1)
        h, u = g * up, up.abs() / power[t]
        u_most = max(u_most, float(u.max()) * 4)
        for r in range(0, H, 4096):
            v = values(w[2][f, r: r + 4096], w[3][f, r: r + 4096])
            out[t, r: r + 4096] += h @ v.T / k
            most[t, r: r + 4096] += u @ v.abs().T
    return out, float(most.max()) * 16, u_most


def _check(case, used=None):
    T, E, k, H, I, form = case
    say("moe exact", case)
    assert moe_form(T, E, k, H, I) == form
    ones = 1 << min(12, int(np.log2(H)))
    w = _weights(E, H, I, k, ones, 1)
    if E * H * I < 1 << 28:
        w = tuple(map(guarded_u8, w))
    x = _activations(T, H, ones, 7)
    rng = np.random.default_rng(3)
    pool = np.arange(E) if used is None else np.array(used)
    chosen = torch.from_numpy(np.stack([rng.permutation(pool)[:k] for _ in range(T)])).to("cuda")
    logits = torch.full((T, E), -200.0, device="cuda").scatter_(1, chosen, 0.0)
    out, ok = guarded((T, H), torch.bfloat16)
    nv.mxfp4_moe(x, logits, *w, k, renormalize=False, out=out)
    exact, steps, u_most = _exact(x, chosen, w, k)
    assert steps < 2.0**24 and u_most < 2.0**16, (steps, u_most)
    want = exact.float().to(torch.bfloat16)
    differ = int((out != want).sum())
    assert differ == 0, f"{differ} of {T * H} outputs are not the rounded exact value"
    assert ok()
    # what the comparison can tell apart: no output at all, and the next expert's
    assert int((want != 0).sum()) > T * H // 2
    if k < E:  # (a token that takes every expert takes the next ones too)
        other = _exact(x, chosen, w, k, 1)[0].float().to(torch.bfloat16)
        apart = int((want != other).sum())
        assert apart > T * H // 2


@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_every_form(case):
    _check(case)


@pytest.mark.parametrize("case", WIDEST, ids=_ids)
def test_widest(case):
    _check(case)


@pytest.mark.parametrize("case", LARGE, ids=_ids)
def test_past_two_to_the_32_bytes(case):
    """512 experts of 8192 x 1024, 4.3 GB of gate and up rows: the first and the last experts chosen."""
    _check(case, used=[0, 1, 255, 256, 510, 511])


def test_most_tokens():
    """2^21 tokens, the largest number taken, as 512 times the same 4096."""
    E, k, H, I = 4, 2, 32, 32
    say("moe exact, most tokens")
    w, x = _weights(E, H, I, k, 32, 1), _activations(4096, H, 32, 7)
    rng = np.random.default_rng(3)
    chosen = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(4096)])).to("cuda")
    logits = torch.full((4096, E), -200.0, device="cuda").scatter_(1, chosen, 0.0)
    logits[::7] = -torch.inf   # tokens without experts
    chosen[::7] = -1
    exact, steps, _ = _exact(x, chosen, w, k)
    assert steps < 2.0**24
    want = exact.float().to(torch.bfloat16)
    out = torch.full((2**21, H), 3.0, dtype=torch.bfloat16, device="cuda")
    nv.mxfp4_moe(x.repeat(512, 1), logits.repeat(512, 1), *w, k, renormalize=False, out=out)
    differ = int((out.view(512, 4096, H) != want).sum())
    assert differ == 0 and not bool(want[::7].any())
