"""The MXFP4 path on the GPU against the oracle.

* Quantization is bit-exact: every bf16 pattern as an element of blocks of many scales,
  constructed ties, clamped exponents, NaN and infinite blocks, ragged shapes; dequantization
  is exact for every code and scale byte.
* The product lies within 2^-10 * sum |a w| + 1 bf16 ulp of the exact value, at sizes that
  reach every kernel, its edges and its ragged parts; scales at both ends of their range.
* linear() equals quantize + gemm bit for bit; streams, captured graphs, empty problems.
"""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import bf16_to_dev, guarded, say, to_host, u8_to_dev
from oracle import mxfp4_oracle as M4
from oracle import nvfp4_oracle as O
from workloads import to_bf16_bits

pytestmark = pytest.mark.gpu


def _check_quantize(bits, label):
    say("mxfp4 quantize", label, bits.shape)
    M, K = bits.shape
    packed, ok_p = guarded((M, K // 2), torch.uint8)
    scales, ok_s = guarded((M, K // 32), torch.uint8)
    nv.mxfp4_quantize(bf16_to_dev(bits), packed, scales)
    wp, ws = M4.quantize(bits)
    gp, gs = to_host(packed), to_host(scales)
    assert np.array_equal(gs, ws), f"{label}: {np.count_nonzero(gs != ws)} scale bytes differ"
    assert np.array_equal(gp, wp), f"{label}: {np.count_nonzero(gp != wp)} code bytes differ"
    assert ok_p() and ok_s(), f"{label}: wrote outside its outputs"


@pytest.mark.parametrize("shape", [(1, 32), (1, 96), (3, 160), (7, 2880), (333, 1440), (64, 4096), (2049, 512)])
def test_quantize_shapes(shape):
    rng = np.random.default_rng(shape[0] * 7 + shape[1])
    x = rng.standard_normal(shape) * np.exp(rng.uniform(-30, 30, (shape[0], 1)))
    _check_quantize(to_bf16_bits(x.astype(np.float32)), "shape")


def test_quantize_every_pattern_at_many_scales():
    """All finite bf16 patterns, 31 to a block behind a leader that sets the block's scale."""
    pats = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    pats = pats[(pats & 0x7F80) != 0x7F80]
    for lead in (0x0001, 0x0080, 0x0100, 0x0180, 0x1000, 0x3F80, 0x40C0, 0x6000, 0x7F7F):
        mine = pats[(pats & 0x7FFF) <= lead]
        mine = np.concatenate([mine, np.zeros(-mine.size % 31, dtype=np.uint16)]).reshape(-1, 31)
        bits = np.concatenate([np.full((mine.shape[0], 1), lead, dtype=np.uint16), mine], axis=1)
        _check_quantize(bits, f"leader {lead:#06x}")


def test_quantize_special_blocks():
    x = np.random.default_rng(3).standard_normal((9, 128)).astype(np.float32)
    x[0, :32], x[1, :32], x[2, :32] = 0.0, -0.0, 2.0**-133
    x[3, 7], x[4, 40], x[5, 127] = np.nan, np.inf, -np.inf
    x[6, :32], x[7, :32] = 3.3e38, 2.0**-126
    _check_quantize(to_bf16_bits(x), "special")
    packed, scales = nv.mxfp4_quantize(bf16_to_dev(to_bf16_bits(x)))
    v = to_host(nv.mxfp4_dequantize(packed, scales).float())
    bad = np.zeros((9, 4), dtype=bool)
    bad[3, 0] = bad[4, 1] = bad[5, 3] = True
    assert np.array_equal(np.isnan(v), np.repeat(bad, 32, axis=1))


def test_dequantize_every_code_and_scale():
    packed = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 256), (256, 1)).reshape(256 * 16, 16)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16).reshape(-1, 1)
    say("mxfp4 dequantize")
    out, ok = guarded((4096, 32), torch.bfloat16)
    got = to_host(nv.mxfp4_dequantize(u8_to_dev(packed), u8_to_dev(scales), out).float()).astype(np.float64)
    want = M4.dequantize(packed, scales)
    want = np.where(np.abs(want) >= 2.0**128, np.sign(want) * np.inf, want)   # beyond bf16
    assert np.array_equal(got, want, equal_nan=True) and ok()


def test_dequantize_ragged():
    rng = np.random.default_rng(8)
    for M, K in ((1, 32), (5, 96), (333, 1440)):
        p = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
        s = rng.integers(1, 250, (M, K // 32), dtype=np.uint8)
        got = to_host(nv.mxfp4_dequantize(u8_to_dev(p), u8_to_dev(s)).float()).astype(np.float64)
        assert np.array_equal(got, M4.dequantize(p, s)), (M, K)


# ---- product --------------------------------------------------------------------------


def _operands(M, N, K, seed, lo=118, hi=131):
    rng = np.random.default_rng(seed)
    return [rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(lo, hi, (M, K // 32), dtype=np.uint8),
            rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(lo, hi, (N, K // 32), dtype=np.uint8)]


def _check_gemm(ops, label, rows=None, cols=None):
    M, N = ops[0].shape[0], ops[2].shape[0]
    say("mxfp4 gemm", label, M, N, 2 * ops[0].shape[1])
    # operands between canary bytes that decode to NaN (scale byte 0xFF): what is read past an end shows
    dev = []
    for a in ops:
        t, _ = guarded(a.shape, torch.uint8, fill=0xFF)
        t.copy_(torch.from_numpy(a))
        dev.append(t)
    out, ok = guarded((M, N), torch.bfloat16)
    nv.mxfp4_gemm(*dev, out=out)
    got = to_host(out)
    assert ok(), f"{label}: wrote outside out"
    r = slice(None) if rows is None else rows
    c = slice(None) if cols is None else cols
    ref, absref = M4.gemm_ref(ops[0][r], ops[1][r], ops[2][c], ops[3][c])
    good, worst, nbad = O.check_gemm(got[r][:, c], ref, absref)
    assert good, f"{label}: {nbad} out of tolerance (worst {worst:.3g})"
    return dev, got


SIZES = [(1, 1, 32), (1, 17, 64), (1, 1000, 96), (1, 4096, 4096), (2, 130, 1440), (5, 33, 288), (16, 257, 512),
         (17, 64, 160), (31, 100, 1024), (32, 512, 2880), (33, 65, 224), (48, 1030, 1056), (64, 64, 8192),
         (65, 129, 736), (100, 300, 320), (127, 255, 256), (128, 128, 128), (129, 1000, 2080), (256, 256, 512),
         (257, 513, 544), (333, 1001, 1440), (512, 640, 1024), (1000, 96, 768),
         (100, 129, 32), (130, 300, 64), (300, 520, 96), (1100, 1030, 480), (2100, 2050, 352), (70, 2000, 448)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_gemm_sizes(size):
    _check_gemm(_operands(*size, seed=sum(size)), "sizes")


@pytest.mark.parametrize("size", [(2048, 2048, 1024), (2600, 1650, 1312), (4608, 9216, 512), (4096, 4097, 2560)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gemm_large_on_sampled_rows_and_columns(size):
    M, N, K = size
    rng = np.random.default_rng(1)
    rows = np.unique(np.concatenate([[0, 1, M - 2, M - 1], rng.integers(0, M, 60)]))
    cols = np.unique(np.concatenate([[0, 1, N - 2, N - 1], rng.integers(0, N, 300)]))
    _check_gemm(_operands(*size, seed=5), "large", rows, cols)


def test_gemm_long_k():
    _check_gemm(_operands(3, 40, 1 << 17, seed=2), "long K")
    _check_gemm(_operands(70, 70, (1 << 15) + 32, seed=3), "long K")


def test_gemm_scale_extremes():
    """Scale bytes at both ends whose product is an ordinary number, and a NaN scale."""
    for size in ((4, 40, 256), (80, 96, 512)):
        M, N, K = size
        ops = _operands(*size, seed=4)
        ops[1][:], ops[3][:] = 0, 252
        _check_gemm(ops, "tiny x huge")
        ops[1][:], ops[3][:] = 250, 3
        _check_gemm(ops, "huge x tiny")
        ops = _operands(*size, seed=4)
        ops[1][1, K // 32 - 1] = 0xFF
        got = to_host(nv.mxfp4_gemm(*map(u8_to_dev, ops)).float())
        assert np.isnan(got[1]).all() and not np.isnan(np.delete(got, 1, axis=0)).any()


@pytest.mark.parametrize("size", [(1, 512, 512), (40, 300, 1440), (300, 520, 2048)], ids=lambda s: "x".join(map(str, s)))
def test_gemm_is_deterministic_and_takes_unaligned_scales(size):
    """The same bits on every call, also with scale tensors that are only 4-byte aligned."""
    ops = _operands(*size, seed=9)
    dev, first = _check_gemm(ops, "determinism")
    moved = []
    for k in (1, 3):
        buf = torch.full((ops[k].size + 8,), 0xFF, dtype=torch.uint8, device="cuda")
        view = buf[4: 4 + ops[k].size].view(ops[k].shape)
        view.copy_(torch.from_numpy(ops[k]))
        moved.append(view)
    for _ in range(3):
        assert np.array_equal(to_host(nv.mxfp4_gemm(dev[0], moved[0], dev[2], moved[1])), first)


# ---- linear, streams, graphs, empties ------------------------------------------------------


LINEAR = [(1, 64, 32), (1, 5120, 5120), (3, 100, 1440), (16, 256, 1024), (17, 300, 2080), (40, 96, 544), (300, 520, 1440)]


def _bf16(M, K, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((M, K), device="cuda", generator=g) * scale).to(torch.bfloat16)


@pytest.mark.parametrize("size", LINEAR, ids=lambda s: "x".join(map(str, s)))
def test_linear_is_quantize_then_gemm(size):
    M, N, K = size
    say("mxfp4 linear", size)
    x, w = _bf16(M, K, 1), nv.mxfp4_quantize(_bf16(N, K, 2, 0.02))
    x[0, 0] = 60.0
    a = nv.mxfp4_quantize(x)
    work, ok = guarded((nv.mxfp4_linear_workspace_bytes(M, K),), torch.uint8)
    got, want = to_host(nv.mxfp4_linear(x, *w, workspace=work)), to_host(nv.mxfp4_gemm(*a, *w))
    assert np.array_equal(got, want) and ok()
    at = (M * K // 2 + 255) // 256 * 256
    assert np.array_equal(to_host(work[: M * K // 2]), to_host(a[0]).reshape(-1))
    assert np.array_equal(to_host(work[at: at + M * K // 32]), to_host(a[1]).reshape(-1))
    ref, absref = M4.gemm_ref(to_host(a[0]), to_host(a[1]), to_host(w[0]), to_host(w[1]))
    assert O.check_gemm(got, ref, absref)[0]


def test_nan_activations_show():
    x, w = _bf16(4, 256, 1), nv.mxfp4_quantize(_bf16(64, 256, 2, 0.1))
    x[2, 100] = float("nan")
    got = to_host(nv.mxfp4_linear(x, *w).float())
    assert np.isnan(got[2]).all() and not np.isnan(got[[0, 1, 3]]).any()


def test_other_stream_and_captured_graph():
    sizes = [(1, 512, 1024), (40, 300, 1440), (200, 256, 512)]
    side = torch.cuda.Stream()
    for M, N, K in sizes:
        say("mxfp4 stream and graph", M, N, K)
        w = nv.mxfp4_quantize(_bf16(N, K, 2, 0.02))
        x = _bf16(M, K, 1)
        want = to_host(nv.mxfp4_linear(x, *w))
        torch.cuda.synchronize()
        got = nv.mxfp4_linear(x, *w, stream=side)
        side.synchronize()
        assert np.array_equal(to_host(got), want)
        # capture quantize -> gemm -> dequantize, replay on new inputs
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        work = torch.empty(nv.mxfp4_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
        back = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        packed, scales = nv.mxfp4_quantize(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.mxfp4_linear(x, *w, out=out, workspace=work)
            nv.mxfp4_quantize(x, packed, scales)
            nv.mxfp4_dequantize(packed, scales, back)
        for seed in (5, 6, 7):
            x.copy_(_bf16(M, K, seed))
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            a = nv.mxfp4_quantize(x)
            assert np.array_equal(to_host(out), to_host(nv.mxfp4_gemm(*a, *w)))
            assert np.array_equal(to_host(back), to_host(nv.mxfp4_dequantize(*a)))


def test_empty_problems():
    e = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    p, s = nv.mxfp4_quantize(e(0, 64, dtype=torch.bfloat16))
    assert p.shape == (0, 32) and s.shape == (0, 2)
    assert nv.mxfp4_dequantize(p, s).shape == (0, 64)
    w = nv.mxfp4_quantize(_bf16(8, 64, 1))
    assert nv.mxfp4_gemm(p, s, *w).shape == (0, 8) and nv.mxfp4_gemm(*w, p, s).shape == (8, 0)
    assert nv.mxfp4_linear(e(0, 64, dtype=torch.bfloat16), *w).shape == (0, 8)
    assert nv.mxfp4_linear(_bf16(3, 64, 1), p, s).shape == (3, 0)


def test_refusals_of_the_binding():
    x, (p, s) = _bf16(4, 64, 1), nv.mxfp4_quantize(_bf16(4, 64, 1))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(_bf16(4, 48, 1))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(x, scales=torch.empty((4, 4), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        nv.mxfp4_gemm(p, s, p[:, :16].contiguous(), s)
    with pytest.raises(ValueError):
        nv.mxfp4_gemm(p.t(), s, p, s)
    with pytest.raises(ValueError):
        nv.mxfp4_dequantize(p, s[:3])
    with pytest.raises(nv.NVFP4Error):
        nv.mxfp4_linear(x, p, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    lib = nv.load_library()
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.nvfp4_mxfp4_gemm(P(p), P(s), P(p), P(s), 4, 4, 64, ctypes.c_void_p(p.data_ptr() + 2), None) == 3
