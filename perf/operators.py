"""Measured cases of the operators around an Engram layer in serving.

Four operators: the wkv projection with the low-rank adapters of many
requests (engram_wkv_adapters), the root-mean-square norm with the residual's
addition and an 8-bit output (engram_norm_quant), beam search's selection over
beams and vocabulary (engram_beam_select), and the reordering of per-beam
states after it (engram_beam_reorder).

``run`` computes them in plain torch operations, or, with ``own`` set, by the
library's entry points.  Sizes are those of the library's own workloads (dim
5120, 4 streams, 24 hash columns of 64, vocabulary 129,280, 4096-token
prefill, 64 sequences in decode, 8 layers) or generic ones.
"""
from __future__ import annotations

import torch

own = False

EPS = 1e-6
HEAD_DIM = 64
E4M3_MAX = 448.0
GROUP = {"e8m0_32": 32, "f32_128": 128, "f32_row": 0}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request decoding one token with its adapter
        dict(name="adapters_decode_1", op="adapters", M=1, dim=5120, hc=4, cols=24, n=4, rank=16, mix="each"),
        # a decode batch of 64 requests, each with its own choice of 32 adapters, some with none
        dict(name="adapters_decode_64", op="adapters", M=64, dim=5120, hc=4, cols=24, n=32, rank=16, mix="each"),
        # a ragged chunk of prompts on a smaller layer
        dict(name="adapters_chunk_613", op="adapters", M=613, dim=2056, hc=2, cols=24, n=5, rank=8, mix="spans"),
        # a whole prefill of eight requests with eight adapters
        dict(name="adapters_prefill_4096", op="adapters", M=4096, dim=5120, hc=4, cols=24, n=8, rank=64, mix="spans"),
        # the four streams of one decoded token
        dict(name="norm_decode_4", op="norm", rows=4, dim=5120, scales="e8m0_32", residual=True),
        # an odd batch, one scale a row, no residual, a width that no group divides
        dict(name="norm_row_1111", op="norm", rows=1111, dim=1032, scales="f32_row", residual=False),
        # the streams of a 4096-token prefill
        dict(name="norm_prefill_16384", op="norm", rows=16384, dim=5120, scales="e8m0_32", residual=True),
        # the first step of one request: only beam 0 is live
        dict(name="beam_first_1x4", op="select", B=1, W=4, V=129280, dtype="float32", first=True),
        # an odd vocabulary: rows at every alignment
        dict(name="beam_odd_7x5", op="select", B=7, W=5, V=32003, dtype="bfloat16", first=False),
        # a decode batch of 64 requests with 8 beams each
        dict(name="beam_decode_64x8", op="select", B=64, W=8, V=129280, dtype="float32", first=False),
        # the look-back of 8 layers follows the beams
        dict(name="reorder_lookback_8", op="reorder", n=8, B=64, W=8, row_bytes=8),
        # large per-beam rows (a running cache of 4 MiB a layer and beam) follow the beams
        dict(name="reorder_rows_4MiB", op="reorder", n=2, B=8, W=8, row_bytes=4 << 20),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("adapters", "norm", "select", "reorder"))
    if op == "adapters":
        rank = rng.choice((8, 16, 24, 32, 64))
        return dict(op=op, M=_spread(rng, 1, 4096), dim=8 * _spread(rng, 32, 640), hc=rng.randint(1, 4),
                    cols=rng.choice((4, 12, 24)), n=rng.randint(1, min(32, 512 // rank)), rank=rank,
                    mix=rng.choice(("each", "spans")))
    if op == "norm":
        return dict(op=op, rows=_spread(rng, 1, 16384), dim=8 * _spread(rng, 16, 640),
                    scales=rng.choice(("e8m0_32", "f32_128", "f32_row")), residual=rng.random() < 0.7)
    if op == "select":
        return dict(op=op, B=_spread(rng, 1, 64), W=rng.randint(1, 8), V=_spread(rng, 1000, 129280),
                    dtype=rng.choice(("float32", "bfloat16")), first=rng.random() < 0.2)
    return dict(op=op, n=rng.randint(1, 8), B=_spread(rng, 1, 64), W=rng.randint(2, 8),
                row_bytes=4 * _spread(rng, 1, 1 << 15))


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    s = dict(case)
    if case["op"] == "adapters":
        K, N, M, n, r = case["cols"] * HEAD_DIM, case["dim"] * (case["hc"] + 1), case["M"], case["n"], case["rank"]
        # table rows: e4m3 normals times a power of two for each block of 32
        e = torch.randint(-4, 5, (M, K // 32, 1), generator=g, device=dev).float()
        rows = torch.randn((M, K // 32, 32), generator=g, device=dev).to(torch.float8_e4m3fn).float()
        s["a"] = (rows * torch.exp2(e)).reshape(M, K).to(torch.bfloat16)
        s["w"] = normal(N, K, std=K ** -0.5)
        s["down"] = normal(n, r, K, std=K ** -0.5)
        s["up"] = normal(n, N, r, std=0.25 * r ** -0.5)
        s["scale"] = 0.5 + torch.rand(n, generator=g, device=dev)
        ids = torch.randint(-1, n, (M,), generator=g, device=dev)
        if case["mix"] == "spans":  # prompts one after the other, each of one request
            ids = torch.sort(ids)[0]
        s["ids"] = ids.to(torch.int32)
    elif case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        s["x"] = normal(rows, dim, std=2.0)
        s["x"][:, 5 % dim] *= 24  # a feature that stands out, as residual streams have
        s["res"] = normal(rows, dim, std=0.5) if case["residual"] else None
        s["weight"] = (1.0 + 0.05 * torch.randn(dim, generator=g, device=dev)).to(torch.bfloat16)
    elif case["op"] == "select":
        B, W, V = case["B"], case["W"], case["V"]
        # beams of one request see nearly the same context; a few tokens stand out
        x = torch.randn((B, 1, V), generator=g, device=dev) * 2
        x = x + 10 * torch.rand((B, 1, V), generator=g, device=dev) ** 24
        x = x + 0.5 * torch.randn((B, W, V), generator=g, device=dev)
        s["logits"] = x.to(getattr(torch, case["dtype"])).reshape(B * W, V)
        cum = -torch.sort(torch.rand((B, W), generator=g, device=dev) * 6 + 2, dim=1)[0]
        if case["first"]:
            cum = torch.full_like(cum, float("-inf"))
            cum[:, 0] = 0.0
        s["cum"] = cum
        fin = torch.rand((B, W), generator=g, device=dev) < 0.1
        s["fin"] = (fin & torch.isfinite(cum)).to(torch.uint8)
        s["eos"], s["pad"] = 1, 0
    else:
        n, B, W, words = case["n"], case["B"], case["W"], case["row_bytes"] // 4
        s["all"] = torch.randint(-(1 << 31), (1 << 31) - 1, (n, B * W, words), generator=g, device=dev,
                                 dtype=torch.int32)
        s["states"] = list(s["all"].unbind(0))
        s["parents"] = torch.randint(0, W, (B, W), generator=g, device=dev, dtype=torch.int32)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return {"adapters": _own_adapters, "norm": _own_norm, "select": _own_select,
                "reorder": _own_reorder}[s["op"]](s)
    return {"adapters": _plain_adapters, "norm": _plain_norm, "select": _plain_select,
            "reorder": _plain_reorder}[s["op"]](s)


def _plain_adapters(s):
    n, r, K = s["down"].shape
    a, M = s["a"].float(), s["a"].shape[0]
    base = a @ s["w"].float().T
    u = (a @ s["down"].float().reshape(n * r, K).T).reshape(M, n, r)
    pick = s["ids"][:, None] == torch.arange(n, device=a.device)
    u = (u * (pick * s["scale"])[:, :, None]).reshape(M, n * r)
    up = s["up"].float().permute(0, 2, 1).reshape(n * r, -1)
    return (base + u @ up).to(torch.bfloat16)


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    rows, dim = y.shape
    group = GROUP[s["scales"]] or dim
    ng = (dim + group - 1) // group
    yg = torch.cat([y, y.new_zeros(rows, ng * group - dim)], 1).reshape(rows, ng, group)
    amax = yg.abs().amax(-1)
    if s["scales"] == "e8m0_32":
        # the smallest power of two that holds the block: amax <= 448 * 2^k, 448 = 0.875 * 2^9
        m, e = torch.frexp(amax)
        k = torch.where(m > 0.875, e - 8, e - 9)
        code = torch.where(amax == 0, torch.zeros_like(k), (k + 127).clamp(0, 254))
        scale = torch.exp2((code - 127).double()).float()
        scales = code.to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        scale = scales = amax / E4M3_MAX
    q = torch.where(scale[:, :, None] > 0, yg / scale[:, :, None], torch.zeros_like(yg))
    q = q.reshape(rows, ng * group)[:, :dim].to(torch.float8_e4m3fn)
    out = {"codes": q, "scales": scales}
    if s["res"] is not None:
        out["sum"] = h.to(torch.bfloat16)
    return out


def _plain_select(s):
    B, W = s["cum"].shape
    x = s["logits"].double().reshape(B, W, -1)  # 64 bits: scores next to each other are told apart
    V = x.shape[2]
    x = x - x.amax(-1, keepdim=True)
    cum = s["cum"].double()[:, :, None]
    score = cum + (x - torch.log(torch.exp(x).sum(-1, keepdim=True)))
    fin = (s["fin"] != 0)[:, :, None]
    is_pad = torch.arange(V, device=x.device) == s["pad"]
    score = torch.where(fin, torch.where(is_pad, cum, float("-inf")), score).reshape(B, W * V)
    best, flat = torch.sort(score, dim=1, descending=True, stable=True)
    best, flat = best[:, :W], flat[:, :W]
    none = best == float("-inf")
    slot = torch.arange(W, device=x.device).expand(B, W)
    parents = torch.where(none, slot, flat // V)
    tokens = torch.where(none, torch.full_like(flat, s["pad"]), flat % V)
    done = torch.gather(s["fin"] != 0, 1, parents) | (tokens == s["eos"])
    return {"tokens": tokens.to(torch.int32), "parents": parents.to(torch.int32), "scores": best.float(),
            "finished": (done & ~none).to(torch.uint8)}


def _plain_reorder(s):
    B, W = s["parents"].shape
    rows = (torch.arange(B, device=s["all"].device)[:, None] * W + s["parents"]).reshape(-1)
    return s["all"].copy_(s["all"][:, rows])


def _kept(s, make):
    """What a serving loop makes once and keeps: the geometry, the adapter set, its output and scratch buffers."""
    if "kept" not in s:
        import gram_memory_layer_amd as ge
        s["kept"] = (ge,) + make(ge)
    return s["kept"]


def _own_adapters(s):
    def make(ge):
        g = ge.Geometry.make(s["dim"], s["hc"], 2, s["cols"], HEAD_DIM, 1, 1)
        ad = ge.Adapters(s["down"], s["up"], s["scale"])
        M, dev = s["a"].shape[0], s["a"].device
        kv = torch.empty((M, g.N), dtype=torch.bfloat16, device=dev)
        scratch = torch.empty(max(ge.engram_wkv_adapters_scratch_size(g, ad, M), 1), dtype=torch.uint8, device=dev)
        return g, ad, kv, scratch
    ge, g, ad, kv, scratch = _kept(s, make)
    return ge.engram_wkv_adapters(g, ad, s["a"], s["w"], s["ids"], kv=kv, scratch=scratch)


def _own_norm(s):
    def make(ge):
        rows, dim, dev = s["x"].shape[0], s["x"].shape[1], s["x"].device
        codes = torch.empty((rows, dim), dtype=torch.uint8, device=dev)
        group = GROUP[s["scales"]] or dim
        kind = torch.uint8 if s["scales"] == "e8m0_32" else torch.float32
        scales = torch.empty((rows, (dim + group - 1) // group), dtype=kind, device=dev)
        return codes, scales, None if s["res"] is None else torch.empty_like(s["x"])
    ge, codes, scales, total = _kept(s, make)
    ge.engram_norm_quant(s["x"], s["weight"], residual=s["res"], eps=EPS, scale_format=s["scales"], codes=codes,
                         scales=scales, total=total)
    if s["scales"] == "e8m0_32":
        scales = scales.view(torch.float8_e8m0fnu)
    out = {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if total is not None:
        out["sum"] = total
    return out


def _own_select(s):
    def make(ge):
        B, W = s["cum"].shape
        dev = s["cum"].device
        out = [torch.empty((B, W), dtype=t, device=dev) for t in (torch.int32, torch.int32, torch.float32, torch.uint8)]
        size = ge.engram_beam_select_scratch_size(B, W, s["logits"].shape[1])
        return out, torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    ge, (tokens, parents, scores, finished), scratch = _kept(s, make)
    ge.engram_beam_select(s["logits"], s["cum"], finished=s["fin"], eos_id=s["eos"], pad_id=s["pad"], tokens=tokens,
                          parents=parents, new_scores=scores, new_finished=finished, scratch=scratch)
    return {"tokens": tokens, "parents": parents, "scores": scores, "finished": finished}


def _own_reorder(s):
    ge, = _kept(s, lambda ge: ())
    ge.engram_beam_reorder(s["states"], s["parents"])
    return s["all"]


# ------------------------------------------------------------------ the floor
def work(case):
    if case["op"] == "adapters":
        K, N, M, n, r = case["cols"] * HEAD_DIM, case["dim"] * (case["hc"] + 1), case["M"], case["n"], case["rank"]
        used = min(n, M)  # adapters that a batch of this size reads
        share = n / (n + 1)  # positions with an adapter
        return {"bytes": 2 * (M * K + N * K + M * N + used * r * (K + N)) + 4 * (M + n),
                "flops": 2 * M * N * K + share * 2 * M * r * (K + N)}
    if case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        group = GROUP[case["scales"]] or dim
        scales = rows * ((dim + group - 1) // group) * (1 if case["scales"] == "e8m0_32" else 4)
        return {"bytes": rows * dim * (3 + (4 if case["residual"] else 0)) + scales + 2 * dim,
                "flops": 6 * rows * dim}
    if case["op"] == "select":
        B, W, V = case["B"], case["W"], case["V"]
        live = B if case["first"] else B * W
        return {"bytes": live * V * (4 if case["dtype"] == "float32" else 2) + B * W * 18, "flops": 4 * live * V}
    n, B, W = case["n"], case["B"], case["W"]
    moved = B * W * (1 - 1 / W)  # rows whose parent is another one, for parents drawn evenly
    read = B * W * (1 - (1 - 1 / W) ** (W - 1))  # rows that another one's parent is
    return {"bytes": n * case["row_bytes"] * (moved + read) + 4 * B * W, "flops": 0}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapters":
        a = s["a"].double()
        out = torch.matmul(a, s["w"].double().transpose(0, 1))
        for j in range(case["n"]):
            at = torch.nonzero(s["ids"] == j).reshape(-1)
            if at.numel():
                low = torch.matmul(a[at], s["down"][j].double().transpose(0, 1))
                out[at] += s["scale"][j].double() * torch.matmul(low, s["up"][j].double().transpose(0, 1))
        return out
    if case["op"] == "norm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        y = h / torch.sqrt(torch.square(h).sum(1, keepdim=True) / case["dim"] + EPS) * s["weight"].double()
        group = GROUP[case["scales"]] or case["dim"]
        blocks = torch.split(y, group, dim=1)
        top = torch.stack([b.abs().max(dim=1).values for b in blocks], 1)
        if case["scales"] == "e8m0_32":
            step = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(-127, 127))
        else:
            step = top / E4M3_MAX
        wide = torch.cat([step[:, i:i + 1].expand(-1, b.shape[1]) for i, b in enumerate(blocks)], 1)
        out = {"codes": torch.where(wide > 0, y / wide, 0.0), "scales": step}
        if s["res"] is not None:
            out["sum"] = h
        return out
    if case["op"] == "select":
        B, W = s["cum"].shape
        per = []
        for b in range(B):
            lp = torch.log_softmax(s["logits"].reshape(B, W, -1)[b].double(), 1) + s["cum"][b].double()[:, None]
            lp = torch.where(s["fin"][b][:, None] != 0, float("-inf"), lp)
            top = torch.topk(lp, W, dim=1).values.reshape(-1)
            ended = torch.where(s["fin"][b] != 0, s["cum"][b].double(), float("-inf"))
            per.append(torch.topk(torch.cat([top, ended]), W).values)
        return {"tokens": None, "parents": None, "scores": torch.stack(per), "finished": None}
    return None
