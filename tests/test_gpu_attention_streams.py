"""Calls that run at the same time, on streams and workspaces of their own: the same bits as one after
another, directly and as branches of one replayed graph."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from attention_parity import Case
from ops_parity import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def work():
    """Attention of one kind and another, their gradients, a norm and clipping: each a function that
    launches on the current stream and returns its outputs."""
    cases = [Case([(700, 900), (130, 2000)], 6, 2, 128, seed=1), Case([(1, 9000), (1, 3)], 5, 1, 64, seed=2),
             Case([(2300, 2300)], 12, 12, 128, seed=3), Case([(60, 60)] * 40, 2, 2, 96, seed=4)]

    def attention(c):
        def run():
            out, lse = B.attention(c.q, c.k, c.v, c.ws, **c.args)
            return [out, lse, *B.attention_bwd(c.q, c.k, c.v, out, lse, c.dout, c.ws, **c.args)]
        return run

    x, res = normal(5, 3000, 1024), normal(6, 3000, 1024)
    grads = [normal(7 + i, 1 << 18) for i in range(30)]
    outs = [torch.empty_like(t) for t in grads]
    ws = B.Workspace(B.grad_clip_workspace_bytes())

    def norm():
        h, rstd, (q, sf) = B.norm_quantize(x, residual=res)
        return [h, rstd, q.view(torch.uint8), sf]

    def clip():
        return [B.grad_clip(grads, 1.0, ws, outs=outs), *outs]

    return [*map(attention, cases), norm, clip], [c.ws for c in cases]


def test_at_the_same_time():
    runs, workspaces = work()
    want = [[t.clone() for t in run()] for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for run, s in zip(runs, streams):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    for ws in workspaces:
        B.check(ws)


def test_as_branches_of_one_graph():
    runs, workspaces = work()
    want = [[t.clone() for t in run()] for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for run, s in zip(runs, streams):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                got.append(run())
        for s in streams:
            main.wait_stream(s)
    for _ in range(5):
        for a in got:
            for t in a:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    for ws in workspaces:
        B.check(ws)
