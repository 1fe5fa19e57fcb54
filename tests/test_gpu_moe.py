"""The mixture-of-experts layer on the GPU against float64.

Router logits to one rounding of the exact sum; the routing's ids exactly; the layer's output
within the bound that the oracle derives from the formula (rounding of h and of the output,
fp32 sums)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host, u8_to_dev
from oracle import mxfp4_oracle as M4

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _guarded_copy(a, fill=0xFF):
    t, _ = guarded(a.shape, torch.uint8, fill=fill)
    t.copy_(torch.from_numpy(a))
    return t


def _experts(E, H, I, seed):
    """Random codes under scales that give outputs of ordinary size, between bytes that read as NaN scales."""
    rng = np.random.default_rng(seed)
    sh = 127 - int(np.log2(H) / 2) - 2
    si = 127 - int(np.log2(I) / 2) - 2
    w = [rng.integers(0, 256, (E, 2 * I, H // 2), dtype=np.uint8),
         rng.integers(sh - 2, sh + 2, (E, 2 * I, H // 32)).astype(np.uint8),
         rng.integers(0, 256, (E, H, I // 2), dtype=np.uint8),
         rng.integers(si - 2, si + 2, (E, H, I // 32)).astype(np.uint8)]
    return w, [_guarded_copy(a) for a in w]


def _check(x, logits, w, dev, top_k, renormalize, label):
    T, H = x.shape
    E, I = w[0].shape[0], 2 * w[2].shape[2]
    say("moe", label, "T", T, "E", E, "k", top_k, "H", H, "I", I, renormalize)
    out, ok = guarded((T, H), torch.bfloat16)
    work, ok_w = guarded((nv.mxfp4_moe_workspace_bytes(T, E, H, I, top_k),), torch.uint8, fill=0xFF)
    _, ids, weights = nv.mxfp4_moe(x, logits, *dev, top_k, renormalize=renormalize, out=out, workspace=work,
                                   return_routing=True)
    wid, wwt = M4.route(to_host(logits), top_k, renormalize)
    assert np.array_equal(to_host(ids), wid), label
    gw = to_host(weights).astype(np.float64)
    assert np.array_equal(np.isnan(gw), np.isnan(wwt))
    fine = ~np.isnan(wwt)
    assert (np.abs(gw - wwt)[fine] <= 2.0**-20 * wwt[fine] + 1e-37).all(), label
    got = to_host(out.float()).astype(np.float64)
    rows = ~np.isnan(wwt).any(axis=1)
    ref, tol = M4.moe_ref(to_host(x.float()).astype(np.float64)[rows], wid[rows], wwt[rows], M4.dequantize(*w[:2]),
                          M4.dequantize(*w[2:]))
    err = np.abs(got[rows] - ref)
    assert (err <= tol + 1e-37).all(), f"{label}: worst {np.nanmax(err / (tol + 1e-37)):.3g} of the bound"
    assert np.isnan(got[~rows]).all()
    assert ok() and ok_w(), f"{label}: wrote outside its buffers"
    return out


CASES = [  # T, E, top_k, H, I
    (1, 1, 1, 32, 32), (1, 4, 2, 64, 96), (1, 60, 6, 512, 352), (2, 8, 8, 96, 160), (3, 5, 2, 224, 64),
    (5, 16, 4, 1024, 480), (12, 32, 4, 640, 288), (16, 128, 8, 512, 128), (17, 7, 3, 160, 224), (31, 64, 8, 256, 256),
    (33, 4, 2, 288, 96), (64, 128, 8, 512, 192), (64, 2, 1, 128, 512), (65, 16, 4, 256, 160), (130, 8, 2, 192, 96),
    (4, 512, 16, 128, 64), (64, 512, 16, 64, 32), (40, 8, 8, 2048, 64), (9, 16, 4, 64, 1440),
    (3, 64, 6, 288, 1408), (4, 32, 8, 96, 544), (2, 40, 16, 4128, 544)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_layer(case):
    T, E, k, H, I = case
    x = _bf16((T, H), sum(case))
    w, dev = _experts(E, H, I, sum(case))
    router = _bf16((E, H), 3, 1.5 / np.sqrt(H))
    logits = nv.moe_router(x, router)
    exact = to_host(x.double()) @ to_host(router.double()).T
    # one rounding to fp32 of a sum that fp64 carries almost exactly
    assert (np.abs(to_host(logits) - exact) <= 2.0**-24 * np.abs(exact) * (1 + 2.0**-20) + 1e-12).all()
    for renormalize in (False, True):
        _check(x, logits, w, dev, k, renormalize, "layer")


@pytest.mark.parametrize("T", [1, 7, 64, 70])
def test_every_token_to_one_expert_and_ties(T):
    E, k, H, I = 8, 2, 128, 96
    x = _bf16((T, H), 1)
    w, dev = _experts(E, H, I, 2)
    l = torch.zeros((T, E), device="cuda")
    _check(x, l, w, dev, k, True, "all equal")              # ties: experts 0 and 1
    l[:, 5], l[:, 3] = 9.0, 8.0
    l[:, 1] = -0.0
    _check(x, l, w, dev, k, False, "one pair")


def test_masked_and_unordered_logits():
    E, k, H, I = 12, 3, 96, 64
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    for T in (10, 64):
        x = _bf16((T, H), 4)
        w, dev = _experts(E, H, I, 5)
        l = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        l[0] = -inf                      # padding: nothing chosen
        l[1, 1:] = -inf                  # one expert only
        l[2] = low                       # the type's lowest value is a value like any other
        l[3, :], l[3, 7] = low, 0.0
        l[4, 4] = nan
        l[5, 2] = inf
        l[6, ::2] = -inf
        l[7] *= 1e30
        l[8] = 3.4e38
        l[9, 0], l[9, 1:] = 88.0, -88.0
        for renormalize in (True, False):
            out = _check(x, l, w, dev, k, renormalize, "masked")
            assert not to_host(out.float())[0].any()


@pytest.mark.parametrize("crowd", [17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("experts", [32, 4])
def test_crowded_experts(crowd, experts):
    """`crowd` of 64 tokens at one expert, the others spread: experts far above the average number of slots, with
    enough rows of weights for the workgroups that stage activations, and experts that all have many."""
    T, k, H, I = 64, 2, 544, 32 * 64 * 17 // experts
    say("crowded", crowd, experts)
    x, (w, dev) = _bf16((T, H), 1), _experts(experts, H, I, 2)
    l = torch.randn((T, experts), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    l[:crowd, experts // 2] = 9.0
    l[crowd:, experts // 2] = -9.0
    _check(x, l, w, dev, k, True, "crowded")


@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 20])
def test_masked_tokens_among_few(T):
    """Masked, short, NaN and infinite rows where every workgroup routes for itself, and around it."""
    E, k, H, I = 12, 3, 96, 64
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    x, (w, dev) = _bf16((T, H), 4), _experts(E, H, I, 5)
    rows = [(slice(None), -inf), (slice(1, None), -inf), (slice(None), low), (4, nan), (2, inf)]
    for first in range(len(rows)):
        l = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(first))
        for t in range(min(T, 4)):
            at, v = rows[(first + t) % len(rows)]
            l[t, at] = v
        for renormalize in (True, False):
            out = to_host(_check(x, l, w, dev, k, renormalize, "masked").float())
            for t in range(min(T, 4)):
                if (first + t) % len(rows) == 0:
                    assert not out[t].any()


@pytest.mark.parametrize("T", [2, 4, 6])
def test_nan_stays_with_its_token_among_few(T):
    E, k, H, I = 6, 2, 160, 64
    x, (w, dev) = _bf16((T, H), 1), _experts(E, H, I, 1)
    l = torch.zeros((T, E), device="cuda")     # all to experts 0 and 1: one tile of columns
    x[1, 150] = float("nan")
    got = to_host(nv.mxfp4_moe(x, l, *dev, k).float())
    assert np.isnan(got[1]).all() and not np.isnan(np.delete(got, 1, axis=0)).any()


def test_every_token_masked():
    x, (w, dev) = _bf16((5, 64), 1), _experts(4, 64, 32, 1)
    l = torch.full((5, 4), -float("inf"), device="cuda")
    out, ids, weights = nv.mxfp4_moe(x, l, *dev, 2, return_routing=True)
    assert not to_host(out.float()).any() and (to_host(ids) == -1).all() and not to_host(weights).any()


def test_nan_stays_with_its_token_and_expert():
    """A NaN activation reaches its own token alone, a NaN scale its expert's tokens alone."""
    T, E, k, H, I = 20, 6, 2, 160, 64
    x, (w, dev) = _bf16((T, H), 1), _experts(E, H, I, 1)
    l = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    ids = M4.route(to_host(l), k, True)[0]
    x[3, 150] = float("nan")
    got = to_host(nv.mxfp4_moe(x, l, *dev, k).float())
    assert np.isnan(got[3]).all() and not np.isnan(np.delete(got, 3, axis=0)).any()
    x[3, 150] = 0.0
    dev[3][2, 17, 1] = 0xFF   # a scale of expert 2's output row 17
    got = to_host(nv.mxfp4_moe(x, l, *dev, k).float())
    hit = (ids == 2).any(axis=1)
    assert np.array_equal(np.isnan(got[:, 17]), hit) and not np.isnan(np.delete(got, 17, axis=1)).any()


@pytest.mark.parametrize("T", [1, 6, 33, 64])
def test_a_token_does_not_depend_on_its_batch(T):
    """A token's routing is that of the token alone, and the same call gives the same bits."""
    E, k, H, I = 16, 4, 512, 224
    x, (w, dev), router = _bf16((T, H), 1), _experts(E, H, I, 3), _bf16((E, H), 3, 0.06)
    l = nv.moe_router(x, router)
    assert np.array_equal(to_host(nv.moe_router(x[T - 1:].contiguous(), router)), to_host(l)[T - 1:])
    first = to_host(nv.mxfp4_moe(x, l, *dev, k))
    for _ in range(3):
        assert np.array_equal(to_host(nv.mxfp4_moe(x, l, *dev, k)), first)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_streams_and_graphs(T):
    """Two streams with workspaces of their own at once, and a captured layer replayed on new inputs."""
    E, k, H, I = 16, 4, 512, 224
    (w, dev), router = _experts(E, H, I, 3), _bf16((E, H), 3, 0.06)
    xs = [_bf16((T, H), s) for s in (1, 2)]
    want = [to_host(nv.mxfp4_moe(x, nv.moe_router(x, router), *dev, k)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            l = nv.moe_router(xs[i], router, stream=st)
            outs[i].append(nv.mxfp4_moe(xs[i], l, *dev, k, stream=st))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o in outs[i]:
            assert np.array_equal(to_host(o), want[i])
    x = xs[0].clone()
    logits = torch.empty((T, E), device="cuda")
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    work = torch.empty(nv.mxfp4_moe_workspace_bytes(T, E, H, I, k), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.moe_router(x, router, logits)
        nv.mxfp4_moe(x, logits, *dev, k, out=out, workspace=work)
    for s in (5, 6, 7):
        x.copy_(_bf16((T, H), s))
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_host(out), to_host(nv.mxfp4_moe(x, nv.moe_router(x, router), *dev, k)))


def test_router_sizes_and_special_values():
    for T, E, H in ((1, 1, 32), (1, 500, 96), (3, 7, 4096), (64, 128, 2048), (131, 33, 160)):
        say("router", T, E, H)
        x, r = _bf16((T, H), T), _bf16((E, H), E)
        out, ok = guarded((T, E), torch.float32)
        got = to_host(nv.moe_router(x, r, out)).astype(np.float64)
        want = to_host(x.double()) @ to_host(r.double()).T
        mag = to_host(x.double().abs()) @ to_host(r.double().abs()).T
        assert (np.abs(got - want) <= 2.0**-24 * np.abs(want) + (H * 2.0**-52) * mag).all() and ok()
    x, r = _bf16((4, 64), 1), _bf16((8, 64), 2)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    got = to_host(nv.moe_router(x, r))
    assert np.isnan(got[1]).all() and np.isinf(got[2]).all() and np.isfinite(got[[0, 3]]).all()


def test_empty_and_refused():
    w, dev = _experts(4, 64, 32, 1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    l = nv.moe_router(x, _bf16((4, 64), 1))
    out, ids, weights = nv.mxfp4_moe(x, l, *dev, 2, return_routing=True)
    assert out.shape == (0, 64) and ids.shape == (0, 2) and weights.shape == (0, 2)
    x = _bf16((3, 64), 1)
    l = nv.moe_router(x, _bf16((4, 64), 1))
    for k in (0, 5, -1):
        with pytest.raises(nv.NVFP4Error):
            nv.mxfp4_moe(x, l, *dev, k)
    with pytest.raises(nv.NVFP4Error):
        nv.mxfp4_moe(x, l, *dev, 2, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        nv.mxfp4_moe(x, l[:, :3].contiguous(), *dev, 2)
    with pytest.raises(TypeError):
        nv.mxfp4_moe(x, l.half(), *dev, 2)
    with pytest.raises(ValueError):
        nv.mxfp4_moe(x, l, dev[0][:, :32].contiguous(), dev[1], dev[2], dev[3], 2)
    with pytest.raises(ValueError):
        nv.moe_router(x, _bf16((4, 96), 1))
