"""The MXFP4 operators as a model's block runs them: a projection, the router, the routed experts,
the residual sum and an output projection, eager and as one captured graph."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import mxfp4_oracle as M4
from oracle import nvfp4_oracle as O

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _quantized(shape, seed, scale):
    """Weights [..., N, K] quantized as the rows of one matrix."""
    p, s = nv.mxfp4_quantize(_bf16((int(np.prod(shape[:-1])), shape[-1]), seed, scale))
    return p.view(*shape[:-1], shape[-1] // 2), s.view(*shape[:-1], shape[-1] // 32)


class Block:
    def __init__(self, T, E, k, H, I, N):
        self.k = k
        self.proj = _quantized((H, H), 1, H**-0.5)
        self.router = _bf16((E, H), 2, 2 * H**-0.5)
        self.w13 = _quantized((E, 2 * I, H), 3, H**-0.5)
        self.w2 = _quantized((E, H, I), 4, I**-0.5)
        self.head = _quantized((N, H), 5, H**-0.5)
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.a, self.moe, self.r, self.y = new(T, H), new(T, H), new(T, H), new(T, N)
        self.logits = new(T, E, dtype=torch.float32)
        bytes_ = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.work = bytes_(nv.mxfp4_linear_workspace_bytes(T, H)), bytes_(nv.mxfp4_moe_workspace_bytes(T, E, H, I, k))

    def __call__(self, x):
        nv.mxfp4_linear(x, *self.proj, out=self.a, workspace=self.work[0])
        nv.moe_router(self.a, self.router, self.logits)
        _, self.ids, self.weights = nv.mxfp4_moe(self.a, self.logits, *self.w13, *self.w2, self.k, renormalize=True,
                                                 out=self.moe, workspace=self.work[1], return_routing=True)
        torch.add(self.a, self.moe, out=self.r)
        nv.mxfp4_linear(self.r, *self.head, out=self.y, workspace=self.work[0])


def _linear_fits(x, w, got):
    a = M4.quantize(to_host(x.view(torch.int16)).view(np.uint16))
    ref, absref = M4.gemm_ref(*a, to_host(w[0]), to_host(w[1]))
    good, worst, nbad = O.check_gemm(to_host(got), ref, absref)
    assert good, f"{nbad} out of tolerance (worst {worst:.3g})"


@pytest.mark.parametrize("T", [1, 4, 9, 23, 66])
def test_block(T):
    """Each step against 64 bits on the step before's output; the graph's replays equal eager runs bit for bit."""
    E, k, H, I, N = 16, 4, 512, 352, 1000
    say("block", T)
    b = Block(T, E, k, H, I, N)
    x = _bf16((T, H), 10 + T)
    b(x)
    torch.cuda.synchronize()
    _linear_fits(x, b.proj, b.a)
    exact = to_host(b.a.double()) @ to_host(b.router.double()).T
    mag = to_host(b.a.double().abs()) @ to_host(b.router.double().abs()).T
    logits = to_host(b.logits)
    assert (np.abs(logits - exact) <= 2.0**-24 * np.abs(exact) + H * 2.0**-52 * mag).all()
    ids, weights = M4.route(logits, k, True)
    assert np.array_equal(to_host(b.ids), ids)
    ref, tol = M4.moe_ref(to_host(b.a.double()), ids, weights, M4.dequantize(*map(to_host, b.w13)),
                          M4.dequantize(*map(to_host, b.w2)))
    assert (np.abs(to_host(b.moe.double()) - ref) <= tol).all()
    _linear_fits(b.r, b.head, b.y)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b(x)
    for seed in (5, 6, 7):
        x.copy_(_bf16((T, H), seed))
        b.y.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        got = to_host(b.y)
        b(x)
        torch.cuda.synchronize()
        assert np.array_equal(got, to_host(b.y))


def test_blocks_on_threads_at_once():
    """Host threads, each with a stream and a block of its own, at once: the bits of a serial run."""
    shapes = [(1, 16, 4, 512, 352, 1000), (4, 8, 2, 288, 96, 64), (17, 16, 4, 512, 352, 200), (70, 32, 8, 256, 64, 33)]
    blocks = [Block(*s) for s in shapes]
    xs = [_bf16((s[0], s[3]), 20 + i) for i, s in enumerate(shapes)]
    want = []
    for b, x in zip(blocks, xs):
        b(x)
        want.append(to_host(b.y).copy())
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    blocks[i].y.fill_(3.0)
                    blocks[i](xs[i])
            st.synchronize()
            if not np.array_equal(blocks[i].y.view(torch.int16).cpu().numpy().view(np.uint16), want[i]):
                bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
