"""The calls at the vocabulary's two ends in a row, as they are used: decode steps that
sample a token, look its row up into the layer's streams and run the layer on
them, and a training step of the embedding through the lookup and its gradient."""
import dataclasses

import pytest
import torch

import synth
from tests import test_gpu_embed, test_gpu_sample
from tests.gpu_util import Workload, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def test_decode_steps_by_sampling(ge):
    dev = torch.device("cuda:0")
    say("vocabulary steps")
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    g, B, V, steps = wl.g, 6, wl.g.vocab, 5
    gen = torch.Generator(device=dev)
    gen.manual_seed(7)
    normal = lambda *s, std=1.0: torch.randn(s, generator=gen, device=dev) * std  # noqa: E731
    table = normal(V, g.dim, std=g.dim ** -0.5).to(torch.bfloat16)
    head = normal(V, g.hc_mult * g.dim, std=0.1).to(torch.bfloat16)
    t = torch.tensor([0.0, 0.7, 1.0, 1.3, 0.9, 1.0], device=dev)
    k = torch.tensor([0, 40, 0, 5, 0, 1], dtype=torch.int32, device=dev)
    p = torch.tensor([1.0, 0.9, 0.95, 1.0, 1.0, 0.5], device=dev)
    m = torch.tensor([0.0, 0.0, 0.05, 0.0, 0.0, 0.0], device=dev)
    start = torch.randint(0, V, (B,), generator=gen, device=dev, dtype=torch.int32)
    us = torch.rand(steps, B, generator=gen, device=dev)

    ids, state = start.clone(), torch.zeros(B, g.max_ngram_size - 1, dtype=torch.int32, device=dev)
    x = torch.empty(B, 1, g.hc_mult, g.dim, dtype=torch.bfloat16, device=dev)
    u, logprobs = us[0].clone(), torch.empty(B, device=dev)
    scratch = torch.empty(ge.engram_sample_scratch_size(B, V), dtype=torch.uint8, device=dev)
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def step():
        ge.engram_embed(table, ids.view(B, 1), scale=g.dim ** 0.5, streams=g.hc_mult, out=x, err=err)
        out = layer.forward(x, ids.view(B, 1), state=state, err=err)
        logits = out.view(B, -1) @ head.t()
        ge.engram_sample(logits, u, temperature=t, top_k=k, top_p=p, min_p=m, tokens=ids, logprobs=logprobs,
                         scratch=scratch, err=err)
        return logits

    seen = []
    for r in range(steps):
        u.copy_(us[r])
        before = ids.clone()
        logits = step()
        want = (table[before.long()].float() * g.dim ** 0.5).to(torch.bfloat16)[:, None, None]
        assert torch.equal(x, want.expand_as(x))
        again, _ = test_gpu_sample.check(ge, logits, u, t, k, p, m)
        assert torch.equal(ids, again)
        seen.append((ids.clone(), logprobs.clone()))
    assert int(err.item()) == 0

    # the same steps from a captured graph
    ids.copy_(start)
    state.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(start)
    state.zero_()
    for r in range(steps):
        u.copy_(us[r])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, seen[r][0]) and torch.equal(logprobs, seen[r][1]), r


def test_a_training_step_of_the_embedding(ge):
    """Two micro-batches of a padded batch: the gradient against the formula's, and the
    loss of the moved table against the one the gradient foretells (linear in the table)."""
    dev = torch.device("cuda:0")
    say("vocabulary training step")
    gen = torch.Generator(device=dev)
    gen.manual_seed(8)
    V, dim, streams, B, T, pad = 1000, 256, 4, 4, 48, 3
    table = torch.randn(V, dim, generator=gen, device=dev)
    grad = None
    target = torch.randn(2, B, T, streams, dim, generator=gen, device=dev)
    ids = torch.randint(0, V, (2, B, T), generator=gen, device=dev, dtype=torch.int32)
    ids[:, :, 30:][torch.rand(2, B, T - 30, generator=gen, device=dev) < 0.5] = pad
    live = (ids != pad)[..., None, None]
    for i in range(2):
        out = ge.engram_embed(table, ids[i], scale=0.5, streams=streams)
        assert out.shape == (B, T, streams, dim)
        grad = ge.engram_embed_grad(target[i], ids[i], V, scale=0.5, pad_id=pad, dtable=grad, accumulate=i > 0)
    every = target.reshape(-1, streams, dim)
    test_gpu_embed.check_grad(grad, every, ids.reshape(-1), V, 0.5, pad=pad)

    def loss(at):
        out = torch.stack([ge.engram_embed(at, ids[i], scale=0.5, streams=streams) for i in range(2)])
        return (out.double() * target * live).sum().item()
    step = torch.randn(V, dim, generator=gen, device=dev)
    moved = loss(table + step) - loss(table)
    told = (grad.double() * ((table + step).double() - table.double())).sum().item()
    # roundings: of each looked-up value and of each gradient's sum of at most a row's terms (2^-24 of
    # the terms' magnitudes), which do not all point one way but are bounded as if they did
    terms = (every.double().abs().sum(1) * 0.5)
    scale = (terms * ((table + step).abs() + table.abs())[ids.reshape(-1).long()].double()).sum().item()
    assert abs(moved - told) <= 2.0 ** -24 * scale * (2 + streams * 64)
