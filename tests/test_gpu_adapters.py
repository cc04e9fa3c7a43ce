"""engram_wkv_adapters and engram_forward_adapted against the formula in 64
bits.

Bound on kv for one element, with S = sum_k |a_k w_k|, D_r = sum_k |down_rk a_k|,
u_r = scale * (down a)_r (all exact), K terms summed in fp32 in any order (each
addition off by at most 2^-23 of what it gives, which also covers a matrix core
that cuts instead of rounding):
  base         (K + 2) 2^-23 S
  u            |scale| (K + 3) 2^-23 D_r, carried into the result by |up_r|
  bf16 pair    2^-16 |u_r|, by |up_r|  (two roundings of 2^-8 each, multiplied)
  second sum   (2 rank + 4) 2^-23 sum_r |up_r u_r|
  bf16         2^-8 of the result, or half a subnormal step 2^-134.
"""
import numpy as np
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


def geometry(ge, dim, hc, cols, head_dim=64):
    return ge.Geometry.make(dim, hc, 2, cols, head_dim, 1, 1)


def reference(a, w, down, up, scale, ids):
    """(kv, bound) in 64 bits."""
    a, w, down, up = (t.double().cpu() for t in (a, w, down, up))
    ids = ids.cpu()
    n, rank, K = down.shape
    scale = torch.ones(n, dtype=torch.float64) if scale is None else scale.double().cpu()
    kv = a @ w.T
    bound = (K + 2) * 2.0 ** -23 * (a.abs() @ w.abs().T)
    for j in range(n):
        at = torch.nonzero(ids == j).reshape(-1)
        if not at.numel():
            continue
        u = scale[j] * (a[at] @ down[j].T)
        du = scale[j].abs() * (K + 3) * 2.0 ** -23 * (a[at].abs() @ down[j].abs().T)
        kv[at] += u @ up[j].T
        bound[at] += (du + (2.0 ** -16 + (2 * rank + 4) * 2.0 ** -23) * (u.abs() + du)) @ up[j].abs().T
    bound += 2.0 ** -8 * (kv.abs() + bound) + 2.0 ** -134
    return kv, bound


def check(kv, ref, bound, what):
    d = (kv.double().cpu() - ref).abs()
    assert torch.isfinite(kv).all(), what
    worst = (d / bound).max().item() if d.numel() else 0.0
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def inputs(dev, M, N, K, n, rank, mix, seed, with_scale=True):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    a, w = r(M, K), r(N, K, std=K ** -0.5)
    down, up = r(n, rank, K, std=K ** -0.5), r(n, N, rank, std=rank ** -0.5)
    scale = torch.rand(n, generator=g, device=dev) * 2 - 0.5 if with_scale else None
    if mix == "none":
        ids = torch.full((M,), -1, device=dev)
    elif mix == "each":
        ids = torch.arange(M, device=dev) % n
    elif mix == "random":
        ids = torch.randint(-1, n, (M,), generator=g, device=dev)
    else:
        ids = torch.sort(torch.randint(-1, n, (M,), generator=g, device=dev))[0]
    return a, w, down, up, scale, ids.to(torch.int32)


CASES = [
    # M, dim, hc, cols, head_dim, n, rank, mix
    (1, 64, 1, 1, 64, 1, 8, "each"), (1, 5120, 4, 24, 64, 4, 16, "each"),
    (2, 72, 2, 3, 32, 3, 16, "random"), (7, 8, 1, 2, 64, 2, 24, "spans"),
    (15, 200, 1, 4, 64, 40, 8, "each"), (16, 264, 1, 24, 64, 16, 32, "each"),
    (17, 264, 2, 12, 64, 5, 40, "random"), (33, 136, 4, 2, 64, 33, 64, "each"),
    (64, 512, 4, 24, 64, 32, 16, "random"), (65, 520, 1, 5, 64, 3, 128, "spans"),
    (96, 104, 3, 1, 32, 7, 16, "none"), (130, 264, 1, 8, 64, 130, 8, "each"),
    (257, 200, 2, 3, 96, 9, 72, "random"), (300, 1032, 1, 24, 64, 6, 64, "spans"),
    (1023, 264, 1, 4, 64, 8, 16, "random"), (1024, 264, 1, 4, 64, 8, 16, "spans"),
    (1300, 1288, 1, 6, 64, 8, 64, "spans"), (1100, 136, 2, 3, 32, 5, 16, "random"),
    # every position its own adapter, at the ranks and batch sizes that share LDS differently
    (64, 136, 1, 4, 64, 64, 128, "each"), (64, 72, 1, 2, 64, 64, 16, "each"),
    (48, 136, 1, 4, 64, 48, 72, "each"), (32, 264, 1, 2, 64, 32, 64, "each"),
    (32, 136, 1, 2, 64, 32, 128, "each"), (16, 72, 1, 2, 64, 16, 128, "each"),
    (9, 72, 1, 2, 64, 16, 48, "each"), (3, 200, 4, 24, 64, 2, 56, "each"),
    # mid-sized batches on both sides of the decode kernel's share of the machine
    (600, 264, 1, 4, 64, 8, 16, "random"), (613, 2056, 2, 24, 64, 5, 8, "spans"),
    (200, 5120, 1, 4, 64, 30, 24, "random"), (400, 5120, 2, 2, 64, 7, 112, "random"),
    # a 128 x 128 tile a compute unit: every count of k-tiles that the ring starts and ends with
    (65, 5120, 4, 1, 64, 3, 16, "spans"), (127, 5120, 4, 2, 64, 4, 40, "random"),
    (128, 5120, 4, 3, 64, 8, 8, "each"), (100, 5120, 4, 4, 64, 2, 128, "random"),
    (81, 5120, 4, 5, 64, 30, 16, "each"), (113, 5120, 4, 6, 64, 5, 72, "spans"),
    (128, 5000, 4, 7, 64, 128, 24, "each"), (90, 5120, 4, 24, 64, 6, 64, "none"),
    (613, 1544, 3, 9, 64, 8, 64, "random"), (512, 1280, 1, 4, 64, 8, 64, "each"),
    # on both sides of the large tiles
    (300, 5120, 4, 2, 64, 5, 16, "random"), (600, 5120, 4, 1, 64, 9, 40, "each"),
    (1030, 2056, 2, 3, 64, 4, 64, "random"), (450, 5000, 4, 3, 64, 450, 8, "each"),
    # more adapters than the order has buckets
    (1500, 136, 1, 2, 64, 2100, 8, "each"), (2100, 136, 1, 2, 64, 2000, 16, "random"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_projection_with_adapters(ge, case):
    M, dim, hc, cols, hd, n, rank, mix = case
    dev = torch.device("cuda:0")
    say("adapters", case)
    g = geometry(ge, dim, hc, cols, hd)
    a, w, down, up, scale, ids = inputs(dev, M, g.N, g.K, n, rank, mix, 11 + M + rank, M % 2 == 0)
    ad = ge.Adapters(down, up, scale)
    # a guard of one row behind the output, and of 256 bytes behind the scratch
    kv = torch.full((M + 1, g.N), 7.0, dtype=torch.bfloat16, device=dev)
    size = ge.engram_wkv_adapters_scratch_size(g, ad, M)
    scratch = torch.full((size + 256,), 255, dtype=torch.uint8, device=dev)  # NaN where not written
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv[:M], scratch=scratch[:size], err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (kv[M] == 7.0).all() and (scratch[size:] == 255).all()
    ref, bound = reference(a, w, down, up, scale, ids)
    check(kv[:M], ref, bound, str(case))
    again = ge.engram_wkv_adapters(g, ad, a, w, ids)
    assert torch.equal(again.view(torch.int16), kv[:M].view(torch.int16))  # the same on every run


@pytest.mark.parametrize("M,dim,hc", [(5, 136, 1), (64, 136, 1), (70, 136, 1), (1050, 136, 1), (100, 5120, 4)])
def test_another_requests_weights_do_not_reach_a_position(ge, M, dim, hc):
    dev = torch.device("cuda:0")
    say("adapter isolation", M, dim, hc)
    g = geometry(ge, dim, hc, 4)
    a, w, down, up, scale, ids = inputs(dev, M, g.N, g.K, 4, 16, "random", 5)
    want = ge.engram_wkv_adapters(g, ge.Adapters(down, up, scale), a, w, ids)
    down, up, a = down.clone(), up.clone(), a.clone()
    down[1] = float("nan")
    up[2] = float("inf")
    at = ids == 3
    a[at] = float("nan")
    got = ge.engram_wkv_adapters(g, ge.Adapters(down, up, scale), a, w, ids)
    keep = (ids == 0) | (ids == -1)
    assert keep.any()
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    assert torch.isnan(got[(ids == 1) | at]).all()


@pytest.mark.parametrize("M", [3, 40, 80, 1030])
def test_ids_outside_count_as_none_and_flag(ge, M):
    dev = torch.device("cuda:0")
    say("adapter ids outside", M)
    g = geometry(ge, 64, 1, 2)
    a, w, down, up, scale, ids = inputs(dev, M, g.N, g.K, 3, 8, "random", 9)
    ad = ge.Adapters(down, up, scale)
    none = ids.clone()
    none[M // 2:] = -1
    bad = ids.clone()
    bad[M // 2:] = torch.tensor([3, -2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev).repeat(
        M)[:M - M // 2]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    want = ge.engram_wkv_adapters(g, ad, a, w, none, err=err)
    assert int(err.item()) == 0
    got = ge.engram_wkv_adapters(g, ad, a, w, bad, err=err)
    assert int(err.item()) == ge.ERRBIT_ADAPTER
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_more_positions_than_one_launch_takes(ge):
    dev = torch.device("cuda:0")
    say("adapters, 262,144 positions and 300 more")
    M = 262144 + 300
    g = geometry(ge, 8, 1, 1)
    a, w, down, up, scale, ids = inputs(dev, M, g.N, g.K, 5, 16, "random", 3)
    kv = ge.engram_wkv_adapters(g, ge.Adapters(down, up, scale), a, w, ids)
    ref, bound = reference(a, w, down, up, scale, ids)
    check(kv, ref, bound, "two launches")


@pytest.mark.parametrize("M", [8, 90000])
def test_offsets_past_32_bits(ge, M):
    dev = torch.device("cuda:0")
    say("adapters far", M)
    g = geometry(ge, 5120, 4, 1)
    # M = 8: 700 adapters whose up rows take 4.6 GB; M = 90000: a result of 4.6 GB
    n, rank = (700, 128) if M == 8 else (6, 16)
    gen = torch.Generator(device=dev)
    gen.manual_seed(M)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    a, w, down = r(M, g.K), r(g.N, g.K, std=g.K ** -0.5), r(n, rank, g.K, std=g.K ** -0.5)
    up = torch.empty(n, g.N, rank, dtype=torch.bfloat16, device=dev)
    for j in range(n):
        up[j] = r(g.N, rank, std=rank ** -0.5)
    ids = (torch.arange(M, device=dev) * 97 + n - 1) % n
    kv = ge.engram_wkv_adapters(g, ge.Adapters(down, up), a, w, ids.to(torch.int32))
    at = torch.arange(M, device=dev) if M == 8 else torch.tensor([0, 1, 41943, 41944, 83885, 83886, 83887, M - 1],
                                                                 device=dev)
    some = ids[at]
    ref, bound = reference(a[at], w, down[some], up[some], None, torch.arange(at.numel()))
    check(kv[at], ref, bound, "far")
    del up, kv
    torch.cuda.empty_cache()


def test_no_positions_and_refusals(ge):
    dev = torch.device("cuda:0")
    g = geometry(ge, 64, 1, 2)
    a, w, down, up, scale, ids = inputs(dev, 4, g.N, g.K, 3, 8, "random", 9)
    ad = ge.Adapters(down, up, scale)
    assert ge.engram_wkv_adapters(g, ad, a[:0], w, ids[:0]).shape == (0, g.N)
    with pytest.raises(ValueError):
        ge.engram_wkv_adapters(g, ad, a, w, ids[:3])
    with pytest.raises(TypeError):
        ge.engram_wkv_adapters(g, ad, a, w, ids.long())
    with pytest.raises(ValueError):
        ge.Adapters(down, up[:2], scale)
    with pytest.raises(ValueError):
        ge.Adapters(down.transpose(1, 2), up, scale)
    with pytest.raises(ValueError):
        ge.engram_wkv_adapters(geometry(ge, 72, 1, 2), ad, a, torch.empty(144, g.K, dtype=a.dtype,
                                                                          device=dev), ids)
    with pytest.raises(ge.EngramError) as e:
        ge.engram_wkv_adapters(g, ad, a, w, ids, scratch=torch.empty(64, dtype=torch.uint8, device=dev))
    assert e.value.status == 3


def test_graph_replays_and_other_streams(ge):
    dev = torch.device("cuda:0")
    say("adapters in a graph")
    g = geometry(ge, 264, 2, 6)
    for M in (4, 40, 200, 1100):
        a, w, down, up, scale, ids = inputs(dev, M, g.N, g.K, 5, 16, "random", 21)
        ad = ge.Adapters(down, up, scale)
        want = ge.engram_wkv_adapters(g, ad, a, w, ids)
        kv = torch.zeros_like(want)
        scratch = torch.empty(ge.engram_wkv_adapters_scratch_size(g, ad, M), dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv, scratch=scratch)
        s.synchronize()
        assert torch.equal(kv, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ge.engram_wkv_adapters(g, ad, a, w, ids, kv=kv, scratch=scratch)
        for r in range(3):
            kv.zero_()
            a.copy_(torch.roll(a, 1, 0))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(kv, ge.engram_wkv_adapters(g, ad, a, w, ids)), (M, r)


@pytest.mark.parametrize("B,T,masked", [(3, 1, False), (2, 9, True), (64, 1, False), (1, 70, True)])
def test_forward_with_adapters_is_its_stages(ge, B, T, masked):
    dev = torch.device("cuda:0")
    say("forward adapted", B, T, masked)
    import dataclasses
    wl = Workload(ge, dataclasses.replace(synth.config("tiny"), head_dim=64), dev)
    g, cfg = wl.g, wl.cfg
    gen = torch.Generator(device=dev)
    gen.manual_seed(B * 100 + T)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    ad = ge.Adapters(r(3, 16, g.K, std=0.1), r(3, g.N, 16, std=0.3))
    aid = torch.arange(B, device=dev, dtype=torch.int32) % 4 - 1
    ids = torch.from_numpy(synth.token_ids(cfg, B, T, name="adapted")).to(dev)
    x = r(B, T, g.hc_mult, g.dim)
    mask = (torch.rand(B, T, generator=gen, device=dev) < 0.7) if masked else None
    state = torch.randint(0, 50, (B, 2), generator=gen, device=dev, dtype=torch.int32)
    st = state.clone()
    gate = torch.empty(B, T, g.hc_mult, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    layer = ge.EngramLayer(g, wl.tables, wl.table, wl.scales, wl.w, wl.q, wl.k)
    out = layer.forward(x, ids, mask=mask, state=st, gate=gate, err=err, adapters=ad, adapter_ids=aid)
    assert int(err.item()) == 0
    st2 = state.clone()
    hid = ge.engram_hash(g, wl.tables, ids, state=st2)
    rows = ge.engram_gather(g, wl.table, wl.scales, hid)
    kv = ge.engram_wkv_adapters(g, ad, rows, wl.w, aid.repeat_interleave(T).contiguous())
    gate2 = torch.empty_like(gate)
    out2 = ge.engram_gate_add(g, x, kv, wl.q, wl.k, mask=mask, gate=gate2)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert torch.equal(gate, gate2) and torch.equal(st, st2)
    ref, bound = reference(rows, wl.w, ad.down, ad.up, None, aid.repeat_interleave(T))
    check(kv, ref, bound, "forward's projection")
    # no adapters at all: the shared projection
    none = torch.full((B,), -1, dtype=torch.int32, device=dev)
    kv0 = ge.engram_wkv_adapters(g, ad, rows, wl.w, none.repeat_interleave(T).contiguous())
    ref, bound = reference(rows, wl.w, ad.down, ad.up, None, none.repeat_interleave(T))
    check(kv0, ref, bound, "no adapters")
    assert np.isfinite(out.float().cpu().numpy()).all()
