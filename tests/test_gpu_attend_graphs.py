"""Captured graphs of dense attention that share workspaces with each other and with eager calls."""

import pytest
import torch

from sparse_linear_attention_sla_b200 import binding
from tests.test_gpu_attend import _make

pytestmark = pytest.mark.gpu


def test_two_graphs_share_workspaces_around_an_eager_call(cuda_device):
    """Two captured graphs of unlike problems on one workspace, replayed in turn with eager calls between them."""
    dev = cuda_device
    data = [_make(21, 1, 4, 2, 1, 2000, 128, dev), _make(22, 1, 2, 2, 260, 260, 64, dev)]
    ps = [binding.attend_problem(q, k, True) for q, k, _, _ in data]
    room = [max((binding.new_workspace_attend(p, dev, back) for p in ps), key=len) for back in (False, True)]

    def step(q, k, v, dO, ws=(None, None)):
        out, lse = binding.attend(q, k, v, causal=True, ws=ws[0])
        return (out, lse) + binding.attend_backward(q, k, v, out, lse, dO, causal=True, ws=ws[1])

    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        for x in data:
            step(*x, ws=room)
    s.synchronize()
    graphs, results = [], []
    for x in data:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(step(*x, ws=room))
        graphs.append(graph)
    for seed in (31, 32):
        shapes = ((1, 4, 2, 1, 2000, 128), (1, 2, 2, 260, 260, 64))
        for x, shape, plus in zip(data, shapes, (0, 5)):
            for dst, src in zip(x, _make(seed + plus, *shape, dev)):
                dst.copy_(src)
        want = []
        for graph, x in zip(graphs, data):
            graph.replay()
            want.append(step(*x, ws=room))
        graphs[0].replay()
        torch.cuda.synchronize(dev)
        binding.check(room[0]), binding.check(room[1])
        for got, ref in zip(results, want):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
