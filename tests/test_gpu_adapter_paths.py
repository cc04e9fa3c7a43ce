"""The kernels that engram_wkv_adapters and engram_forward_adapted choose between,
each at sizes that reach it: against the formula in 64 bits (bounds as in
test_gpu_adapters), ids that are no adapter's, another request's NaN and
infinity, other streams and replayed graphs.

`way` states the library's rules once more, so that a size which no longer
reaches its kernel fails here."""
import dataclasses

import pytest
import torch

import synth
from tests.gpu_util import Workload, say
from tests.test_gpu_adapters import check, geometry, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def way(M, N, K, rank):
    """(the second product's kernel, whether the positions are ordered first, the first product's ranks at once)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    up = lambda a, b: -(-a // b)  # noqa: E731
    rt = up(rank, 16)
    tiles = lambda t: up(M, t) * up(N, t)  # noqa: E731
    down = 1 if rt == 1 or M <= 1024 else 2 if rt == 2 else 4
    if K % 64 == 0 and (M <= 64 or tiles(64) <= (1 if rank > 32 and M >= 256 else 2) * cus):
        return "rows", False, down
    first = M * rt > 1536
    if K % 64:
        return "general 256" if M >= 1024 else "general 64", first, down
    if tiles(128) <= cus:
        return "ring", first, down
    if 2 * up(tiles(128), cus) <= 5 * up(tiles(256), cus):
        return "tiles 128", first, down
    tm, nb = up(M, 256), up(N, 256)
    if tm * nb % cus:
        whole = [c for c in range(nb - 1, 0, -1) if tm * c % cus == 0]
        if whole and up(M, 128) * up(N - whole[0] * 256, 128) <= cus:
            return "tiles 256 and 128", first, down
    return "tiles 256", first, down


def case_inputs(ge, dev, M, dim, hc, cols, hd, n, rank, mix, seed):
    g = geometry(ge, dim, hc, cols, hd)
    return g, inputs(dev, M, g.N, g.K, n, rank, mix, seed)


FORMULA = [
    # M, dim, hc, cols, head_dim, n, rank, mix, way
    (4096, 5120, 4, 1, 64, 8, 64, "random", ("tiles 256 and 128", True, 4)),
    (4096, 5120, 4, 2, 64, 3, 128, "spans", ("tiles 256 and 128", True, 4)),
    (4091, 5120, 4, 1, 64, 33, 24, "random", ("tiles 256 and 128", True, 2)),
    (300, 5120, 4, 1, 64, 5, 64, "random", ("tiles 256", False, 1)),
    (300, 5120, 4, 3, 64, 7, 128, "each", ("tiles 256", True, 1)),
    (300, 5120, 4, 2, 64, 300, 24, "each", ("tiles 256", False, 1)),
    (271, 5000, 4, 1, 64, 4, 72, "spans", ("tiles 256", False, 1)),
    (600, 5120, 4, 2, 64, 9, 128, "random", ("tiles 128", True, 1)),
    (600, 5120, 4, 1, 64, 6, 72, "each", ("tiles 128", True, 1)),
    (200, 2560, 3, 5, 64, 6, 128, "random", ("ring", True, 1)),
    (1100, 2056, 1, 2, 64, 5, 24, "random", ("tiles 128", True, 2)),
    (1700, 264, 1, 3, 64, 7, 32, "each", ("rows", False, 2)),
    (2100, 136, 1, 2, 64, 40, 40, "random", ("rows", False, 4)),
    (1300, 264, 1, 2, 64, 5, 72, "spans", ("rows", False, 4)),
    (2011, 520, 1, 1, 64, 9, 128, "random", ("ring", True, 4)),
    (1030, 2056, 2, 2, 64, 6, 128, "each", ("tiles 128", True, 4)),
    (700, 520, 1, 3, 32, 5, 64, "random", ("general 64", True, 1)),
    (1500, 520, 1, 3, 32, 6, 128, "random", ("general 256", True, 4)),
    (1100, 520, 1, 1, 32, 6, 24, "each", ("general 256", True, 2)),
]


@pytest.mark.parametrize("case", FORMULA, ids=lambda c: "-".join(str(v) for v in c[:-1]))
def test_formula(ge, case):
    M, dim, hc, cols, hd, n, rank, mix, want = case
    dev = torch.device("cuda:0")
    say("adapter path", case)
    g, (a, w, down, up, scale, ids) = case_inputs(ge, dev, M, dim, hc, cols, hd, n, rank, mix, M + rank)
    assert way(M, g.N, g.K, rank) == want
    ad = ge.Adapters(down, up, scale)
    kv = torch.full((M + 1, g.N), 7.0, dtype=torch.bfloat16, device=dev)
    size = ge.engram_wkv_adapters_scratch_size(g, ad, M)
    scratch = torch.full((size + 256,), 255, dtype=torch.uint8, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv[:M], scratch=scratch[:size], err=err)
    assert int(err.item()) == 0
    assert (kv[M] == 7.0).all() and (scratch[size:] == 255).all()
    # all columns of some rows: the first and last, and those around every 128th
    rows = torch.cat([torch.arange(0, M, 128), torch.arange(127, M, 128),
                      torch.randperm(M, generator=torch.Generator().manual_seed(M))[:100], torch.tensor([M - 1])])
    rows = torch.unique(rows).to(dev)
    ref, bound = reference(a[rows], w, down, up, scale, ids[rows])
    check(kv[rows], ref, bound, str(case))
    assert torch.isfinite(kv).all()
    again = ge.engram_wkv_adapters(g, ad, a, w, ids)
    assert torch.equal(again.view(torch.int16), kv[:M].view(torch.int16))


PATHS = [
    # M, dim, hc, cols, head_dim, rank, way
    (40, 264, 2, 4, 64, 16, ("rows", False, 1)),
    (1100, 136, 1, 2, 64, 24, ("rows", False, 2)),
    (100, 5120, 4, 1, 64, 16, ("ring", False, 1)),
    (200, 2560, 3, 2, 64, 128, ("ring", True, 1)),
    (300, 5120, 4, 1, 64, 16, ("tiles 256", False, 1)),
    (300, 5120, 4, 1, 64, 128, ("tiles 256", True, 1)),
    (600, 5120, 4, 1, 64, 8, ("tiles 128", False, 1)),
    (600, 5120, 4, 1, 64, 64, ("tiles 128", True, 1)),
    (4096, 5120, 4, 1, 64, 16, ("tiles 256 and 128", True, 1)),
    (700, 520, 1, 3, 32, 16, ("general 64", False, 1)),
    (700, 520, 1, 3, 32, 64, ("general 64", True, 1)),
    (1500, 520, 1, 3, 32, 8, ("general 256", False, 1)),
    (1100, 520, 1, 3, 32, 40, ("general 256", True, 4)),
]
path_ids = lambda c: "-".join(str(v) for v in c[:-1])  # noqa: E731


def same(p, q):
    return torch.equal(p.view(torch.int16), q.view(torch.int16))


@pytest.mark.parametrize("case", PATHS, ids=path_ids)
def test_another_requests_weights_do_not_reach_a_position(ge, case):
    M, dim, hc, cols, hd, rank, want = case
    dev = torch.device("cuda:0")
    say("adapter path, isolation", case)
    g, (a, w, down, up, scale, ids) = case_inputs(ge, dev, M, dim, hc, cols, hd, 4, rank, "random", 5)
    assert way(M, g.N, g.K, rank) == want
    clean = ge.engram_wkv_adapters(g, ge.Adapters(down, up, scale), a, w, ids)
    down, up, a = down.clone(), up.clone(), a.clone()
    down[1] = float("nan")
    up[2] = float("inf")
    at = ids == 3
    a[at] = float("nan")
    got = ge.engram_wkv_adapters(g, ge.Adapters(down, up, scale), a, w, ids)
    keep = (ids == 0) | (ids == -1)
    assert keep.any()
    assert same(got[keep], clean[keep])
    assert torch.isnan(got[(ids == 1) | at]).all() and not torch.isfinite(got[ids == 2]).any()


@pytest.mark.parametrize("case", PATHS, ids=path_ids)
def test_ids_outside_count_as_none_and_flag(ge, case):
    M, dim, hc, cols, hd, rank, want = case
    dev = torch.device("cuda:0")
    say("adapter path, ids outside", case)
    g, (a, w, down, up, scale, ids) = case_inputs(ge, dev, M, dim, hc, cols, hd, 3, rank, "random", 9)
    assert way(M, g.N, g.K, rank) == want
    ad = ge.Adapters(down, up, scale)
    outside = torch.tensor([3, -2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    # half of them, and a single one in the last place
    for at in (torch.arange(M // 2, M, device=dev), torch.tensor([M - 1], device=dev)):
        none, bad = ids.clone(), ids.clone()
        none[at] = -1
        bad[at] = outside.repeat(M)[:at.numel()]
        err.zero_()
        clean = ge.engram_wkv_adapters(g, ad, a, w, none, err=err)
        assert int(err.item()) == 0
        got = ge.engram_wkv_adapters(g, ad, a, w, bad, err=err)
        assert int(err.item()) == ge.ERRBIT_ADAPTER
        assert same(got, clean)
        assert same(ge.engram_wkv_adapters(g, ad, a, w, bad), clean)  # without a flag


@pytest.mark.parametrize("case", PATHS, ids=path_ids)
def test_graph_replays_and_other_streams(ge, case):
    M, dim, hc, cols, hd, rank, want = case
    dev = torch.device("cuda:0")
    say("adapter path, graph", case)
    g, (a, w, down, up, scale, ids) = case_inputs(ge, dev, M, dim, hc, cols, hd, 5, rank, "random", 21)
    assert way(M, g.N, g.K, rank) == want
    ad = ge.Adapters(down, up, scale)
    eager = ge.engram_wkv_adapters(g, ad, a, w, ids)
    kv = torch.zeros_like(eager)
    scratch = torch.empty(ge.engram_wkv_adapters_scratch_size(g, ad, M), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv, scratch=scratch)
    s.synchronize()
    assert same(kv, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv, scratch=scratch)
    for r in range(3):
        kv.zero_()
        a.copy_(torch.roll(a, 1, 0))
        ids.copy_(torch.roll(ids, 7, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert same(kv, ge.engram_wkv_adapters(g, ad, a, w, ids)), r


@pytest.mark.parametrize("B,T,rank,masked,want", [
    (64, 1, 16, False, ("rows", False, 1)), (1, 100, 16, True, ("ring", False, 1)),
    (3, 100, 64, False, ("tiles 256", False, 1)), (5, 127, 16, True, ("tiles 128", False, 1)),
    (8, 512, 64, True, ("tiles 256 and 128", True, 4)), (9, 455, 16, False, ("tiles 256 and 128", True, 1))])
def test_forward_of_full_size(ge, B, T, rank, masked, want):
    """The layer's full width (1536 -> 25,600), hashed into a small table: the forward
    bit for bit its stages, their projection against the formula, state and masks."""
    dev = torch.device("cuda:0")
    say("forward adapted, full width", B, T, rank, masked)
    tiny = synth.config("tiny")
    wl = Workload(ge, dataclasses.replace(tiny, dim=5120, hc_mult=4, n_heads=24 // (tiny.max_ngram_size - 1),
                                          head_dim=64), dev)
    g, cfg = wl.g, wl.cfg
    assert (g.K, g.N) == (1536, 25600) and way(B * T, g.N, g.K, rank) == want
    gen = torch.Generator(device=dev)
    gen.manual_seed(B * 1000 + T)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    n = 7
    ad = ge.Adapters(r(n, rank, g.K, std=0.03), r(n, g.N, rank, std=0.3),
                     torch.rand(n, generator=gen, device=dev) + 0.5)
    aid = torch.arange(B, device=dev, dtype=torch.int32) % (n + 1) - 1
    aid = aid[torch.randperm(B, generator=gen, device=dev)].contiguous()
    ids = torch.from_numpy(synth.token_ids(cfg, B, T, name="adapted_full")).to(dev)
    x = r(B, T, g.hc_mult, g.dim)
    mask = (torch.rand(B, T, generator=gen, device=dev) < 0.7) if masked else None
    state = torch.randint(0, 50, (B, g.max_ngram_size - 1), generator=gen, device=dev, dtype=torch.int32)
    st, gate, err = state.clone(), torch.empty(B, T, g.hc_mult, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    out = layer.forward(x, ids, mask=mask, state=st, gate=gate, err=err, adapters=ad, adapter_ids=aid)
    assert int(err.item()) == 0
    st2, gate2, each = state.clone(), torch.empty_like(gate), aid.repeat_interleave(T).contiguous()
    rows = ge.engram_gather(g, wl.table, wl.scales, ge.engram_hash(g, wl.tables, ids, state=st2))
    kv = ge.engram_wkv_adapters(g, ad, rows, wl.w, each)
    out2 = ge.engram_gate_add(g, x, kv, wl.q, wl.k, mask=mask, gate=gate2)
    assert same(out, out2) and torch.equal(gate, gate2) and torch.equal(st, st2)
    if masked:
        assert same(out[~mask], x[~mask])
    at = torch.unique(torch.cat([torch.arange(0, B * T, max(B * T // 60, 1)), torch.tensor([B * T - 1])])).to(dev)
    ref, bound = reference(rows.reshape(B * T, -1)[at], wl.w, ad.down, ad.up, ad.scale, each[at])
    check(kv.reshape(B * T, -1)[at], ref, bound, "projection")
    # ids that are no adapter's, over the sequences
    bad = torch.where(aid < 0, torch.full_like(aid, n), aid)
    if (aid < 0).any():
        again = layer.forward(x, ids, mask=mask, state=state.clone(), err=err, adapters=ad, adapter_ids=bad)
        assert int(err.item()) == ge.ERRBIT_ADAPTER and same(again, out)
