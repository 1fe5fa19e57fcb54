"""The fused residual and norm on the GPU against 64 bits, within the bounds counted in
oracle/block_oracle.py; its quantized results byte for byte against the quantizers."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import guarded, say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _bf16(shape, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale + shift).to(torch.bfloat16)


def _f64(t):
    return None if t is None else to_host(t.float()).astype(np.float64)


def _bits(t):
    return t.view(torch.int16)


def _parts(M, H, G, which, seed):
    """The optional operands that `which` names."""
    make = {"weight": lambda i: _bf16((H,), i, 0.3, 1.0), "bias": lambda i: _bf16((H,), i, 0.3),
            "post_weight": lambda i: _bf16((H,), i, 0.3, 0.5), "gate": lambda i: _bf16((G, H), i),
            "scale": lambda i: _bf16((G, H), i, 0.3), "shift": lambda i: _bf16((G, H), i, 0.3)}
    return {name: make[name](seed + i) for i, name in enumerate(make) if name in which}


def _reference(x, y, kind, parts, group, c=1.0, eps=EPS, got_h=None):
    """(h, its tolerance, n of the h that was stored, its tolerance); group [M], -1: none."""
    p = {k: _f64(v) for k, v in parts.items()}
    rows = {k: np.where((group >= 0)[:, None], p[k][np.maximum(group, 0)], 0.0) for k in ("gate", "scale", "shift") if k in p}
    if y is None:
        h, ht = _f64(x), 0.0
    else:
        h, ht = BO.residual(_f64(x), _f64(y), kind, eps, p.get("post_weight"), rows.get("gate"), c)
    n, nt = BO.normed(_f64(x) if got_h is None else _f64(got_h), kind, eps, p.get("weight"), p.get("bias"), rows.get("scale"),
                      rows.get("shift"))
    return h, ht, n, nt


def _check(M, H, G, kind, which, rows=None, c=1.0, seed=0, x=None, y=None, eps=EPS):
    say("add_norm", M, H, G, kind, *which)
    branch = "y" in which
    x = _bf16((M, H), seed + 20, 1.5, 0.25) if x is None else x
    y = (_bf16((M, H), seed + 21, 2.0, -0.5) if y is None else y) if branch else None
    parts = _parts(M, H, G, which, seed)
    out, ok = guarded((M, H), torch.bfloat16)
    h, ok_h = guarded((M, H), torch.bfloat16) if branch else (None, lambda: True)
    before = x.clone()
    got_h, got = nv.add_norm(x, y, kind=kind, rows=rows, residual_scale=c, eps=eps, h=h, out=out, **parts)
    assert ok() and ok_h() and torch.equal(_bits(x), _bits(before))
    assert (got_h is h) if branch else (got_h is x)
    group = to_host(rows).astype(np.int64) if rows is not None else np.arange(M) // max(M // G, 1)
    group = np.where((group >= 0) & (group < G), group, -1)
    rh, ht, rn, nt = _reference(x, y, kind, parts, group, c, eps, got_h)
    if branch:
        keep = (group < 0) & ("gate" in parts)
        err = np.abs(_f64(got_h) - rh)[~keep]
        assert (err <= ht[~keep]).all(), f"h: worst {np.max(err / ht[~keep]):.3g} of the bound"
        assert torch.equal(_bits(got_h)[torch.from_numpy(keep).cuda()], _bits(x)[torch.from_numpy(keep).cuda()])
    err = np.abs(_f64(got) - rn)
    assert (err <= nt).all(), f"n: worst {np.max(err / nt):.3g} of the bound"
    if branch:  # in place
        x2 = x.clone()
        a, b = nv.add_norm(x2, y, kind=kind, rows=rows, residual_scale=c, eps=eps, h=x2, **parts)
        assert a is x2 and torch.equal(_bits(a), _bits(got_h)) and torch.equal(_bits(b), _bits(got))
    return x, y, parts, got_h, got


WIDTHS = [8, 16, 72, 504, 512, 520, 1000, 1024, 1032, 1160, 2048, 2056, 4096, 4104, 6144, 6152, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, kind):
    _check(5, H, 1, kind, ("y", "weight"), seed=H)
    _check(6, H, 3, kind, ("y", "weight", "bias", "post_weight", "gate", "scale", "shift"), seed=H, c=0.5)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("which", [(), ("weight",), ("weight", "bias"), ("scale", "shift"), ("scale",), ("shift",), ("y",), ("y", "gate"),
                                   ("y", "post_weight"), ("y", "post_weight", "gate"), ("y", "gate", "scale", "shift"),
                                   ("bias", "scale")], ids=lambda w: "+".join(w) or "plain")
def test_parts(which, kind):
    for M, H, G in ((1, 264, 1), (12, 264, 4), (12, 1544, 12), (35, 640, 5)):
        _check(M, H, G, kind, which, seed=M + H)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 63, 257, 1025, 5000])
def test_rows(M):
    for H in (64, 2304):
        _check(M, H, 1, "rms", ("y", "weight"), seed=M)
        _check(M, H, M, "layer", ("y", "gate", "scale", "shift"), seed=M)


@pytest.mark.parametrize("H", [72, 1536, 9000])
def test_groups_in_any_order(H):
    M, G = 23, 4
    rows = torch.from_numpy(np.random.default_rng(H).integers(-2, G + 2, M).astype(np.int32)).cuda()
    rows[0], rows[1], rows[2] = 2**31 - 1, -(2**31), G - 1
    for which in (("y", "gate", "scale", "shift"), ("y", "scale"), ("scale", "shift", "weight"), ("y", "weight")):
        for kind in ("rms", "layer"):
            _check(M, H, G, kind, which, rows=rows, seed=H)


@pytest.mark.parametrize("H", [64, 1160, 4096])
def test_extreme_rows(H):
    """Rows far from zero, all alike, zero, tiny and huge ones."""
    for kind in ("rms", "layer"):
        x, y = _bf16((8, H), 1), _bf16((8, H), 2)
        x[0], y[0] = 0.0, 0.0
        x[1], y[1] = 1000.0, 0.0                    # no variance
        x[2] = (1000.0 + 8.0 * x[2].float()).to(torch.bfloat16)
        x[3], y[3] = (x[3].float() * 1e-6).to(torch.bfloat16), 0.0   # below eps
        x[4] = (x[4].float() * 1e15).to(torch.bfloat16)
        y[5] = (y[5].float() * 1e15).to(torch.bfloat16)
        x[6], x[6, 3] = 0.0, 1.0
        _check(8, H, 1, kind, ("y", "weight"), seed=3, x=x, y=y)
        _check(8, H, 1, kind, ("y", "post_weight", "weight"), seed=3, x=x, y=y)
        _check(8, H, 1, kind, ("weight",), seed=3, x=x, eps=1e-3)


def test_nan_and_infinities_stay_in_their_row():
    M, H = 9, 520
    x, y = _bf16((M, H), 1), _bf16((M, H), 2)
    w = _bf16((H,), 3)
    clean = nv.add_norm(x, y, weight=w)
    x[4, 7], y[5, 100], x[6, 1] = float("nan"), float("inf"), -float("inf")
    h, n = nv.add_norm(x, y, weight=w)
    rows = [0, 1, 2, 3, 7, 8]
    assert torch.equal(_bits(h[rows]), _bits(clean[0][rows])) and torch.equal(_bits(n[rows]), _bits(clean[1][rows]))
    assert torch.isnan(n[4]).all() and torch.isnan(n[5, 100]) and h[5, 100] == float("inf") and h[6, 1] == -float("inf")
    # a row that is not modulated keeps x whatever its branch holds
    rows = torch.tensor([0, 0, 0, 0, 0, -1, 0, 0, 0], dtype=torch.int32, device="cuda")
    h, _ = nv.add_norm(x, y, weight=w, gate=_bf16((1, H), 4), rows=rows)
    assert torch.equal(_bits(h[5]), _bits(x[5]))


def _quantizers(gs):
    return {"nvfp4": lambda n: nv.quantize(n, gs), "mxfp4": nv.mxfp4_quantize, "mxfp8": nv.mxfp8_quantize, "fp8r": nv.fp8r_quantize}


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8", "fp8r"])
@pytest.mark.parametrize("H", [32, 96, 512, 544, 1056, 2048, 2080, 4128, 6176, 8192, 8224, 16416, 32768])
def test_quantized_results_are_the_quantizers(H, fmt):
    for M, kind, which in ((7, "rms", ("y", "weight")), (6, "layer", ("y", "post_weight", "gate", "scale", "shift")), (1, "rms", ())):
        say("quantized", fmt, M, H, kind)
        x, y, parts, h, n = _check(M, H, 1, kind, which, seed=H)
        x[M - 1] = 0.0
        if y is not None:
            y[M - 1] = 0.0
        h, n = nv.add_norm(x, y, kind=kind, **parts)
        scales = [0.01, nv.calibrate_device(n), 1e-4] if fmt == "nvfp4" else [None]  # 1e-4: block scales saturate
        for gs in scales:
            q = _quantizers(gs)[fmt](n)
            codes, ok_c = guarded(q[0].shape, torch.uint8)
            sc, ok_s = guarded(q[1].shape, q[1].dtype)
            h2, got = nv.add_norm(x, y, kind=kind, quantize=fmt, global_scale=gs, out=codes, scales=sc, **parts)
            assert got[0] is codes and got[1] is sc and ok_c() and ok_s()
            assert torch.equal(_bits(h2), _bits(h))
            assert torch.equal(codes, q[0]) and torch.equal(sc.view(torch.uint8), q[1].view(torch.uint8))


def test_quantized_many_rows_and_bad_blocks():
    M, H = 3000, 1056
    x, y, w = _bf16((M, H), 1, 3.0), _bf16((M, H), 2), _bf16((H,), 3)
    x[5, 40], x[6, 41] = float("nan"), float("inf")
    _, n = nv.add_norm(x, y, weight=w)
    for fmt in ("mxfp4",):
        _, got = nv.add_norm(x, y, weight=w, quantize=fmt)
        want = _quantizers(None)[fmt](n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_far_rows():
    """Tensors past 2^31 elements."""
    M, H = 2**19 + 5, 4096
    x = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    x[-3:], y[-3:] = _bf16((3, H), 1), _bf16((3, H), 2)
    w = _bf16((H,), 3)
    h, n = nv.add_norm(x, y, weight=w, h=x)
    want = nv.add_norm(_bf16((3, H), 1), _bf16((3, H), 2), weight=w)
    assert torch.equal(_bits(h[-3:]), _bits(want[0])) and torch.equal(_bits(n[-3:]), _bits(want[1]))
    assert not n[:-3].any()


def test_empty():
    x = _bf16((0, 64), 1)
    h, n = nv.add_norm(x, x.clone(), weight=_bf16((64,), 2))
    assert h.shape == n.shape == (0, 64)
    _, (codes, scales) = nv.add_norm(x, quantize="mxfp4")
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


def test_refusals():
    x, y, w, g = _bf16((4, 64), 1), _bf16((4, 64), 2), _bf16((64,), 3), _bf16((2, 64), 4)
    for bad in (dict(weight=w[:32]), dict(bias=g), dict(gate=g), dict(post_weight=w), dict(h=x), dict(kind="batch"),
                dict(y=y[:2]), dict(y=y, gate=g, scale=g[:1]), dict(y=y, gate=g[:, :32].contiguous()), dict(quantize="int8"),
                dict(rows=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(global_scale=1.0), dict(quantize="mxfp4", global_scale=1.0),
                dict(scales=w), dict(out=y[:2]), dict(y=y.t()), dict(weight=w.cpu()),
                dict(quantize="mxfp4", out=torch.empty((4, 64), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            nv.add_norm(x, **bad)
    for bad in (dict(weight=w.float()), dict(y=y.half()), dict(rows=torch.zeros(4, device="cuda")), dict(quantize="nvfp4"),
                dict(quantize="mxfp4", out=y)):
        with pytest.raises(TypeError):
            nv.add_norm(x, **bad)
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(scale=_bf16((3, 64), 1)), dict(quantize="nvfp4", global_scale=-1.0)):
        with pytest.raises(nv.NVFP4Error):
            nv.add_norm(x, **bad)
    with pytest.raises(nv.NVFP4Error):
        nv.add_norm(_bf16((4, 12), 1))
    with pytest.raises(ValueError):
        nv.add_norm(_bf16((4, 48), 1), quantize="mxfp8")
