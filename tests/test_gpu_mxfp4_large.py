"""MXFP4 operators on tensors whose offsets pass 2^31 and 2^32, checked on sampled rows."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import mxfp4_oracle as M4
from oracle import nvfp4_oracle as O

pytestmark = pytest.mark.gpu


def _u8(shape, seed, lo=0, hi=256):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)


def _at(t, rows):
    return to_host(t[torch.as_tensor(rows, device="cuda")])


def test_quantize_and_back():
    M, K = 70001, 32768
    say("mxfp4 quantize", M, K)
    x = _u8((M, 2 * K), 1, 0, 0x7F).view(torch.bfloat16)
    p, s = nv.mxfp4_quantize(x)
    back = nv.mxfp4_dequantize(p, s)
    rows = [0, 1, 32767, 32768, 65535, 65536, 65537, M - 2, M - 1]
    wp, ws = M4.quantize(_at(x.view(torch.int16), rows).view(np.uint16))
    assert np.array_equal(_at(p, rows), wp) and np.array_equal(_at(s, rows), ws)
    assert np.array_equal(to_host(back[torch.as_tensor(rows, device="cuda")].double()), M4.dequantize(wp, ws))


@pytest.mark.parametrize("size", [(3, 140003, 32768), (140003, 3, 32768), (70001, 32769, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gemm(size):
    M, N, K = size
    say("mxfp4 gemm", size)
    a, w = (_u8((M, K // 2), 1), _u8((M, K // 32), 2, 118, 131)), (_u8((N, K // 2), 3), _u8((N, K // 32), 4, 118, 131))
    out = nv.mxfp4_gemm(*a, *w)
    pick = lambda n: list(range(n)) if n < 16 else [0, 1, n // 2, n * 15 // 16, n - 3, n - 2, n - 1]  # noqa: E731
    r, c = pick(M), pick(N)
    ref, absref = M4.gemm_ref(_at(a[0], r), _at(a[1], r), _at(w[0], c), _at(w[1], c))
    got = to_host(out[torch.as_tensor(r, device="cuda")][:, torch.as_tensor(c, device="cuda")].contiguous())
    good, worst, nbad = O.check_gemm(got, ref, absref)
    assert good, f"{nbad} out of tolerance (worst {worst:.3g})"


@pytest.mark.parametrize("T", [2, 6, 20])
def test_moe(T):
    """512 experts of 8192 x 1024: 4.3 GB of gate and up rows; the first and the last experts chosen."""
    E, k, H, I = 512, 2, 8192, 1024
    say("moe", T)
    w = (_u8((E, 2 * I, H // 2), 1), _u8((E, 2 * I, H // 32), 2, 117, 121),
         _u8((E, H, I // 2), 3), _u8((E, H, I // 32), 4, 119, 123))
    used = [0, 255, 510, 511]
    logits = torch.full((T, E), -torch.inf, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(T)
    logits[:, used] = torch.randn((T, len(used)), device="cuda", generator=g)
    x = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
    out, ids, _ = nv.mxfp4_moe(x, logits, *w, k, renormalize=True, return_routing=True)
    wid, wwt = M4.route(to_host(logits), k, True)
    assert np.array_equal(to_host(ids), wid)
    few = [_at(t, used) for t in w]
    ref, tol = M4.moe_ref(to_host(x.double()), np.searchsorted(used, wid), wwt, M4.dequantize(*few[:2]),
                          M4.dequantize(*few[2:]))
    assert (np.abs(to_host(out.double()) - ref) <= tol).all()


@pytest.mark.parametrize("M", [2, 70])
def test_gemm_at_the_longest_k(M):
    K, N = 2**22, 5
    say("mxfp4 gemm, longest K", M)
    a, w = (_u8((M, K // 2), 1), _u8((M, K // 32), 2, 118, 131)), (_u8((N, K // 2), 3), _u8((N, K // 32), 4, 118, 131))
    r = [0, M - 1]
    ref, absref = M4.gemm_ref(_at(a[0], r), _at(a[1], r), to_host(w[0]), to_host(w[1]))
    good, worst, nbad = O.check_gemm(to_host(nv.mxfp4_gemm(*a, *w))[r], ref, absref)
    assert good, f"{nbad} out of tolerance (worst {worst:.3g})"


@pytest.mark.parametrize("case", [(3, 2**20, 32), (6, 2**20, 32), (2, 32, 2**20), (6, 32, 2**20)],
                         ids=lambda c: "x".join(map(str, c)))
def test_moe_at_the_widest(case):
    T, H, I = case
    say("moe, widest", case)
    sh, si = (109, 127) if H > I else (126, 109)   # scales that give sums of ordinary size
    w = (_u8((1, 2 * I, H // 2), 1), _u8((1, 2 * I, H // 32), 2, sh, sh + 3),
         _u8((1, H, I // 2), 3), _u8((1, H, I // 32), 4, si, si + 3))
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
    out = nv.mxfp4_moe(x, torch.zeros((T, 1), device="cuda"), *w, 1)
    ref, tol = M4.moe_ref(to_host(x.double()), np.zeros((T, 1), dtype=np.int32), np.ones((T, 1)),
                          M4.dequantize(*map(to_host, w[:2])), M4.dequantize(*map(to_host, w[2:])))
    assert (np.abs(to_host(out.double()) - ref) <= tol).all()


def test_router_of_many_tokens():
    T, E, H = 270001, 5, 32
    x = _u8((T, 2 * H), 1, 0, 0x40).view(torch.bfloat16)
    w = torch.randn((E, H), device="cuda").to(torch.bfloat16)
    got, want = nv.moe_router(x, w).double(), x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    assert bool(((got - want).abs() <= 2.0**-24 * want.abs() + H * 2.0**-52 * mag).all())
