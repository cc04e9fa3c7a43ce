"""EngramLayer's workspace beside captured graphs: a graph keeps the one it was
captured with when a larger call makes the layer take another."""
import dataclasses

import pytest
import torch

import synth
from tests.gpu_util import Workload, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


@pytest.mark.parametrize("adapted", [False, True])
def test_a_graph_keeps_its_workspace(ge, adapted):
    dev = torch.device("cuda:0")
    say("layer workspace, adapters", adapted)
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    g, B = wl.g, 3
    gen = torch.Generator(device=dev)
    gen.manual_seed(4)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    kw = {}
    if adapted:
        kw = dict(adapters=ge.Adapters(r(2, 8, g.K, std=0.1), r(2, g.N, 8, std=0.3)),
                  adapter_ids=torch.tensor([1, -1, 0], dtype=torch.int32, device=dev))
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    ids = torch.from_numpy(synth.token_ids(wl.cfg, B, 1, name="one")).to(dev)
    x, out = r(B, 1, g.hc_mult, g.dim), torch.empty(B, 1, g.hc_mult, g.dim, dtype=torch.bfloat16, device=dev)
    layer.forward(x, ids, out=out, **kw)
    small = layer._ws
    at, size = small.data_ptr(), small.numel()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, ids, out=out, **kw)
    assert layer._ws is small
    del small
    many = torch.from_numpy(synth.token_ids(wl.cfg, B, 300, name="many")).to(dev)
    xm = r(B, 300, g.hc_mult, g.dim)
    layer.forward(xm, many, **kw)
    assert layer._ws.numel() > size
    # nothing that is allocated now lies where the graph writes
    other = [torch.full((size,), 0x5A, dtype=torch.uint8, device=dev) for _ in range(4)]
    assert all(t.data_ptr() + size <= at or at + size <= t.data_ptr() for t in other)
    for k in range(3):
        x.copy_(torch.roll(x, 1, 0))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = layer.forward(x, ids, **kw)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), k
        assert all(bool((t == 0x5A).all()) for t in other), k


def test_one_that_no_graph_has_is_given_back(ge):
    dev = torch.device("cuda:0")
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    layer = ge.EngramLayer(wl.g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    for n in (1, 100, 5000):
        layer.workspace(n)
    assert layer._kept == [] and layer._ws.numel() == ge.engram_forward_workspace_size(wl.g, 5000)
