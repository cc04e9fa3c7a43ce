"""The serving calls in a row, as a decode loop runs them: the forward with each
request's adapter, the norm into the next product's 8-bit input, a product to
logits, beam selection, the look-back states reordered, the chosen tokens into
the next step."""
import dataclasses

import pytest
import torch

import synth
from tests import test_gpu_adapters, test_gpu_beam, test_gpu_norm_quant
from tests.gpu_util import Workload, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def test_decode_steps_with_adapters_and_beams(ge):
    dev = torch.device("cuda:0")
    say("serving steps")
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    g = wl.g
    B, W, V, steps = 3, 4, g.vocab, 5
    gen = torch.Generator(device=dev)
    gen.manual_seed(77)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    ad = ge.Adapters(r(2, 8, g.K, std=0.1), r(2, g.N, 8, std=0.3), torch.tensor([0.5, 2.0], device=dev))
    request = torch.tensor([0, -1, 1], dtype=torch.int32, device=dev)  # adapter of each request
    aid = request.repeat_interleave(W).contiguous()
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    embed, head = r(V, g.hc_mult, g.dim), r(V, g.hc_mult * g.dim, std=(g.hc_mult * g.dim) ** -0.5)
    norm_w = r(g.dim, std=0.1) + 1

    prompt = torch.from_numpy(synth.token_ids(wl.cfg, B, 6, name="beams")).to(dev)
    n = g.max_ngram_size - 1
    # two layers' look-back; the second hashes the same ids with the same tables
    states = [torch.zeros(B * W, n, dtype=torch.int32, device=dev) for _ in range(2)]
    first = prompt.repeat_interleave(W, 0).contiguous()
    for st in states:
        ge.engram_hash(g, wl.tables, first[:, :-1].contiguous(), state=st)
    history = first.view(B, W, -1)
    ids = first[:, -1:].contiguous()
    scores = torch.full((B, W), float("-inf"), device=dev)
    scores[:, 0] = 0
    finished = torch.zeros(B, W, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    for step in range(steps):
        x = embed[ids.reshape(-1).long()].view(B * W, 1, g.hc_mult, g.dim)
        ge.engram_hash(g, wl.tables, ids, state=states[1], err=err)
        out = layer.forward(x, ids, state=states[0], err=err, adapters=ad, adapter_ids=aid)
        total = torch.empty_like(out)
        codes, scales, _ = ge.engram_norm_quant(out, norm_w, residual=x, total=total)
        test_gpu_norm_quant.check(out, x, norm_w, 1e-6, "e8m0_32", codes, scales, total)
        deq = codes.view(torch.float8_e4m3fn).float().view(B * W, -1, 32) * torch.exp2(
            scales.float().view(B * W, -1, 1) - 127)
        logits = deq.view(B * W, -1) @ head.float().T
        args = (logits, scores.clone(), finished.clone(), 3, 0)
        tokens, parents, scores, finished = ge.engram_beam_select(
            logits, scores, finished=finished, eos_id=3, new_scores=scores, new_finished=finished, err=err)
        test_gpu_beam.check((tokens, parents, scores, finished), *args)
        ge.engram_beam_reorder(states, parents, err=err)
        history = torch.cat([torch.gather(history, 1, parents.long()[:, :, None].expand_as(history)),
                             tokens[:, :, None]], 2)
        ids = tokens.reshape(-1, 1).contiguous()
        # the carried look-back is that of each beam's own history
        fresh = torch.zeros_like(states[0])
        ge.engram_hash(g, wl.tables, history[:, :, :-1].reshape(B * W, -1).contiguous(), state=fresh)
        assert torch.equal(states[0], fresh) and torch.equal(states[1], fresh), step
    assert int(err.item()) == 0
    rows = ge.engram_gather(g, wl.table, wl.scales, ge.engram_hash(g, wl.tables, ids))
    kv = ge.engram_wkv_adapters(g, ad, rows, wl.w, aid)
    ref, bound = test_gpu_adapters.reference(rows, wl.w, ad.down, ad.up, ad.scale, aid)
    test_gpu_adapters.check(kv, ref, bound, "last step")


def test_a_captured_step_replays_as_the_eager_one(ge):
    dev = torch.device("cuda:0")
    say("serving step in a graph")
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    g = wl.g
    B, W, V = 2, 3, g.vocab
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    ad = ge.Adapters(r(2, 8, g.K, std=0.1), r(2, g.N, 8, std=0.3))
    aid = torch.tensor([0, 0, 0, 1, 1, 1], dtype=torch.int32, device=dev)
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    x, logits = r(B * W, 1, g.hc_mult, g.dim), torch.randn(B * W, V, generator=gen, device=dev)
    ids = torch.from_numpy(synth.token_ids(wl.cfg, B * W, 1, name="graph")).to(dev)
    state0 = torch.randint(0, 50, (B * W, 2), generator=gen, device=dev, dtype=torch.int32)
    scores0 = -torch.rand(B, W, generator=gen, device=dev)

    def step(state, scores, ids):
        out = layer.forward(x, ids, state=state, adapters=ad, adapter_ids=aid)
        codes, scales, total = ge.engram_norm_quant(out, residual=x)
        tokens, parents, _, fin = ge.engram_beam_select(logits, scores, new_scores=scores)
        ge.engram_beam_reorder([state], parents)
        ids.copy_(tokens.view(-1, 1))
        return out, codes, scales, total, tokens, parents, fin

    eager_state, eager_scores, eager_ids = state0.clone(), scores0.clone(), ids.clone()
    step(eager_state.clone(), eager_scores.clone(), eager_ids.clone())
    state, scores, gids = state0.clone(), scores0.clone(), ids.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(state, scores, gids)
    state.copy_(state0)
    scores.copy_(scores0)
    gids.copy_(ids)
    for k in range(4):
        logits.copy_(torch.roll(logits, 31, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager_state, eager_scores, eager_ids)
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want)), k
        assert torch.equal(state, eager_state) and torch.equal(scores, eager_scores), k
        assert torch.equal(gids, eager_ids), k
