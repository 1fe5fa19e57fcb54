"""The operators around a block's linears as a transformer block runs them: norm into MXFP4, projection, adapters,
gated residual and norm, router, routing, the routed experts and the next residual; eager, as captured graphs (two at
once on one workspace among them), on other streams and on host threads at once."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say, to_host
from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale + shift).to(torch.bfloat16)


def _quantized(shape, seed, scale):
    p, s = nv.mxfp4_quantize(_bf16((int(np.prod(shape[:-1])), shape[-1]), seed, scale))
    return p.view(*shape[:-1], shape[-1] // 2), s.view(*shape[:-1], shape[-1] // 32)


class Block:
    """T tokens in two sequences, H wide."""

    def __init__(self, T, E, k, H, I, R=16, L=3):
        self.k, self.E = k, E
        self.w1, self.w2, self.post = (_bf16((H,), i, 0.2, 1.0) for i in (1, 2, 3))
        self.gate, self.scale, self.shift = (_bf16((2, H), i, 0.3) for i in (4, 5, 6))
        self.rows = (torch.arange(T, device="cuda") >= (T + 1) // 3).to(torch.int32)
        self.proj = _quantized((H, H), 7, H**-0.5)
        self.a, self.b = _bf16((L, R, H), 8, H**-0.5), _bf16((L, H, R), 9, R**-0.5)
        self.adapters = torch.arange(T, device="cuda", dtype=torch.int32) % (L + 1) - 1
        self.router, self.bias = _bf16((E, H), 10, 2 * H**-0.5), _bf16((E,), 11, 0.05).float()
        self.e13, self.e2 = _quantized((E, 2 * I, H), 12, H**-0.5), _quantized((E, H, I), 13, I**-0.5)

    def __call__(self, x):
        _, q = nv.add_norm(x, weight=self.w1, quantize="mxfp4")
        y = nv.mxfp4_gemm(*q, *self.proj)
        y = nv.lora(y, x, self.a, self.b, self.adapters, out=y)
        h, n = nv.add_norm(x, y, weight=self.w2, gate=self.gate, scale=self.scale, shift=self.shift, rows=self.rows)
        logits = nv.moe_router(n, self.router)
        ids, weights = nv.moe_route(logits, self.k, bias=self.bias, scores="sigmoid", groups=4, top_groups=2, group_best=2)
        m = nv.mxfp4_moe_routed(n, ids, weights, *self.e13, *self.e2)
        out, last = nv.add_norm(h, m, post_weight=self.post, weight=self.w1, kind="layer", h=h)
        return {"y": y, "n": n, "ids": ids, "weights": weights, "m": m, "out": out, "last": last}


def _same(a, b):
    return all(torch.equal(a[k].view(torch.int16), b[k].view(torch.int16)) for k in a)


SHAPES = [(1, 16, 4, 512, 352), (4, 8, 2, 288, 96), (17, 16, 4, 512, 64), (70, 32, 8, 256, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_block_and_its_graph(shape):
    say("block", *shape)
    T, H = shape[0], shape[3]
    b, x = Block(*shape), _bf16((T, H), 20)
    r = b(x)
    torch.cuda.synchronize()
    # spot checks of the chain: the routing of its own logits, the last norm of its own stream
    logits = nv.moe_router(r["n"], b.router)
    ids, w = BO.route(to_host(logits), b.k, to_host(b.bias), "sigmoid", 4, 2, 2)
    assert np.array_equal(to_host(r["ids"]), ids) and (np.abs(to_host(r["weights"]) - w) <= BO.route_tol(w)).all()
    n, tol = BO.normed(to_host(r["out"].double()), "layer", 1e-6, to_host(b.w1.double()))
    assert (np.abs(to_host(r["last"].double()) - n) <= tol).all()
    assert torch.isfinite(r["last"].float()).all()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = b(x)
    for seed in (5, 6, 7):
        x.copy_(_bf16((T, H), seed))
        for t in captured.values():
            t.view(torch.int16).fill_(3)
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in captured.items()}
        assert _same(got, b(x)), seed
        torch.cuda.synchronize()


def test_two_graphs_share_workspaces():
    """Replays in either order, with eager calls between them, on workspaces that both graphs and these use."""
    T, N, K, R, L, E, H, I, k = 20, 130, 256, 16, 4, 16, 256, 64, 4
    y, x, a, b = _bf16((T, N), 1), _bf16((T, K), 2), _bf16((L, R, K), 3, 0.1), _bf16((L, N, R), 4)
    ad = torch.arange(T, device="cuda", dtype=torch.int32) % L
    e13, e2 = _quantized((E, 2 * I, H), 5, 0.1), _quantized((E, H, I), 6, 0.1)
    work = torch.empty(max(nv.lora_workspace_bytes(T, N, K, R), nv.mxfp4_moe_workspace_bytes(T, E, H, I, k)),
                       dtype=torch.uint8, device="cuda")
    l = torch.randn((T, E), device="cuda")

    def one():
        return nv.lora(y, x, a, b, ad, workspace=work)

    def two():
        return nv.mxfp4_moe_routed(x, *nv.moe_route(l, k), *e13, *e2, workspace=work)

    graphs, outs = [], []
    for f in (one, two):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for i, order in enumerate(((0, 1), (1, 0), (0, 0, 1), (1, 1, 0))):
        x.copy_(_bf16((T, K), 30 + i))
        l.normal_()
        want = [one().clone(), two().clone()]
        for o in outs:
            o.zero_()
        for j in order:
            graphs[j].replay()
            work.fill_(0xFF)
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), w.view(torch.int16)) for o, w in zip(outs, want)), order


def test_streams():
    """`stream=` launches and allocates there; a stream of another device is refused."""
    T, N, K, R, L = 300, 520, 256, 16, 4
    y, x, a, b = _bf16((T, N), 1), _bf16((T, K), 2), _bf16((L, R, K), 3, 0.1), _bf16((L, N, R), 4)
    ad = torch.arange(T, device="cuda", dtype=torch.int32) % L
    l = torch.randn((T, 64), device="cuda")
    want = nv.lora(y, x, a, b, ad), *nv.moe_route(l, 6), *nv.add_norm(x, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nv.lora(y, x, a, b, ad, stream=s), *nv.moe_route(l, 6, stream=s), *nv.add_norm(x, x, stream=s)
    _, q = nv.add_norm(x, x, quantize="mxfp4", stream=s)
    s.synchronize()
    assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(got, want))
    assert torch.equal(nv.mxfp4_quantize(want[-1])[0], q[0])


def test_blocks_on_threads_at_once():
    blocks = [Block(*s) for s in SHAPES]
    xs = [_bf16((s[0], s[3]), 20 + i) for i, s in enumerate(SHAPES)]
    want = [b(x) for b, x in zip(blocks, xs)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                got = [blocks[i](xs[i]) for _ in range(15)]
            st.synchronize()
            bad.extend(i for g in got if not _same(g, want[i]))
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(SHAPES))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not any(t.is_alive() for t in threads) and not bad, bad
