"""Low-rank adapters whose first product goes through the workspace: captured graphs, two of them on one workspace, a block's graph,
and blocks on host threads at once."""
import threading

import pytest
import torch

import nvfp4_block_scaled_02_amd as nv
from gpu_helpers import say
from test_gpu_block_run import Block, _bf16, _same

pytestmark = pytest.mark.gpu

# T, N, K, R, L: one fragment of ranks per workgroup, two, many rows at once with v shared
FORMS = [(20, 130, 256, 40, 4), (300, 520, 256, 16, 4), (1999, 264, 136, 64, 5), (4500, 200, 72, 96, 3)]
BLOCKS = [(17, 16, 4, 512, 64), (70, 32, 8, 256, 64)]


def _call(T, N, K, R, L, seed, work):
    y, x, a, b = _bf16((T, N), seed), _bf16((T, K), seed + 1), _bf16((L, R, K), seed + 2, 0.1), _bf16((L, N, R), seed + 3)
    ad = torch.arange(T, device="cuda", dtype=torch.int32) % (L + 1) - 1
    return x, lambda: nv.lora(y, x, a, b, ad, workspace=work)


@pytest.mark.parametrize("first", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_two_graphs_share_a_workspace(first):
    """Replays in either order, with eager calls and the workspace overwritten between them."""
    say("graphs", *first)
    second = FORMS[(FORMS.index(first) + 1) % len(FORMS)]
    sizes = [nv.lora_workspace_bytes(*f[:4]) for f in (first, second)]
    assert min(sizes) > 0
    work = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    calls = [_call(*f, 10 * i, work) for i, f in enumerate((first, second))]
    graphs, outs = [], []
    for _, f in calls:
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for i, order in enumerate(((0, 1), (1, 0), (0, 0, 1), (1, 1, 0))):
        for x, _ in calls:
            x.copy_(_bf16(tuple(x.shape), 30 + i))
        want = [f().clone() for _, f in calls]
        for o in outs:
            o.zero_()
        for j in order:
            graphs[j].replay()
            work.fill_(0xFF)
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), w.view(torch.int16)) for o, w in zip(outs, want)), order


def _block(shape):
    T, H = shape[0], shape[3]
    assert nv.lora_workspace_bytes(T, H, H, 64) > 0
    return Block(*shape, R=64, L=5), _bf16((T, H), 20)


@pytest.mark.parametrize("shape", BLOCKS, ids=lambda s: "x".join(map(str, s)))
def test_block_and_its_graph(shape):
    say("block", *shape)
    b, x = _block(shape)
    b(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = b(x)
    for seed in (5, 6, 7):
        x.copy_(_bf16(tuple(x.shape), seed))
        for t in captured.values():
            t.view(torch.int16).fill_(3)
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in captured.items()}
        assert _same(got, b(x)), seed
        torch.cuda.synchronize()


def test_on_threads_at_once():
    """Each with workspaces of its own."""
    say("threads")
    runs = [(b, x, b(x)) for b, x in map(_block, BLOCKS)]
    calls = [_call(*f, 7 * i, None) for i, f in enumerate(FORMS)]
    runs += [(lambda _, f=f: {"out": f()}, None, {"out": f()}) for _, f in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        f, x, want = runs[i]
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                got = [f(x) for _ in range(15)]
            st.synchronize()
            bad.extend(i for g in got if not _same(g, want))
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not any(t.is_alive() for t in threads) and not bad, bad
