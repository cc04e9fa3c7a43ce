"""Measured cases of the vocabulary's two ends beside an Engram layer.

Three operators: the choice of the next token from given random numbers under
temperature, top-k, top-p and min-p (engram_sample), the lookup of embedding
rows with a scale into the layer's streams (engram_embed), and the gradient of
that lookup (engram_embed_grad).

``run`` computes them in plain torch operations, or, with ``own`` set, by the
library's entry points.  Sizes are those of the library's own workloads (dim
5120, 4 streams, 24 hash columns of 64, vocabulary 129,280, 4096-token
prefill, 64 sequences in decode, 32,768 positions of Zipf ids) or generic ones.
"""
from __future__ import annotations

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request decoding one token, all filters on
        dict(name="sample_decode_1", op="sample", B=1, V=129280, dtype="float32", temp="one", k=50, p=0.95, m=0.0),
        # an odd batch over an odd vocabulary (rows at every alignment); requests of all kinds, greedy ones among them
        dict(name="sample_odd_7", op="sample", B=7, V=32003, dtype="bfloat16", temp="mixed", k=-1, p=-1.0, m=-1.0),
        # a decode batch of 64 requests with top-p: flat rows keep thousands of tokens, peaked ones a few
        dict(name="sample_decode_64", op="sample", B=64, V=129280, dtype="float32", temp="mixed", k=0, p=0.9, m=0.0),
        # rollouts: 512 sequences at a temperature, no filter
        dict(name="sample_rollout_512", op="sample", B=512, V=129280, dtype="bfloat16", temp="one", k=0, p=1.0, m=0.0),
        # a decode step's tokens into the layer's four streams
        dict(name="embed_decode_64", op="embed", n=64, rows=129280, dim=5120, streams=4, table="bfloat16",
             out="bfloat16", ids="even"),
        # a ragged chunk's 24 hash columns from trained fp32 rows of 64
        dict(name="embed_hash_rows_14712", op="embed", n=14712, rows=1 << 20, dim=64, streams=1, table="float32",
             out="bfloat16", ids="even"),
        # a prefill's tokens into the four streams
        dict(name="embed_prefill_4096", op="embed", n=4096, rows=129280, dim=5120, streams=4, table="bfloat16",
             out="bfloat16", ids="zipf"),
        # the tiny layer's step: 16 positions, 4 streams, vocabulary 1000
        dict(name="grad_tiny_16", op="grad", n=16, rows=1000, dim=256, streams=4, grad="float32", table="float32",
             ids="even", add=False),
        # an odd number of positions over an odd vocabulary, a bf16 gradient of a padded batch
        dict(name="grad_odd_1111", op="grad", n=1111, rows=32003, dim=1032, streams=1, grad="bfloat16",
             table="bfloat16", ids="padded", add=False),
        # a 4096-token step of the four streams into the whole vocabulary's gradient
        dict(name="grad_tokens_4096", op="grad", n=4096, rows=129280, dim=5120, streams=4, grad="bfloat16",
             table="float32", ids="zipf", add=False),
        # a long sequence's tokens added to a gradient that is there (micro-batches): a few ids take most positions
        dict(name="grad_long_32768", op="grad", n=32768, rows=129280, dim=2056, streams=1, grad="bfloat16",
             table="float32", ids="zipf", add=True),
        # the 24 hash columns of a 4096-token step into rows of 64
        dict(name="grad_hash_rows_98304", op="grad", n=98304, rows=1 << 20, dim=64, streams=1, grad="bfloat16",
             table="float32", ids="even", add=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("sample", "embed", "grad"))
    if op == "sample":
        return dict(op=op, B=_spread(rng, 1, 256), V=_spread(rng, 1000, 129280),
                    dtype=rng.choice(("float32", "bfloat16")), temp=rng.choice(("one", "mixed")),
                    k=rng.choice((0, 0, _spread(rng, 1, 1000), -1)), p=rng.choice((1.0, 0.8, 0.9, 0.95, -1.0)),
                    m=rng.choice((0.0, 0.0, 0.02, 0.1, -1.0)))
    dim, streams = 8 * _spread(rng, 1, 640), rng.randint(1, 4)
    n = _spread(rng, 1, max(1, min(98304, (4096 * 4 * 5120) // (dim * streams))))
    rows = _spread(rng, 1000, min(1 << 20, (129280 * 5120) // dim))
    kinds = ("float32", "bfloat16")
    ids = rng.choice(("even", "zipf", "padded"))
    if op == "embed":
        return dict(op=op, n=n, rows=rows, dim=dim, streams=streams, table=rng.choice(kinds), out=rng.choice(kinds),
                    ids=ids)
    return dict(op=op, n=n, rows=rows, dim=dim, streams=streams, grad=rng.choice(kinds), table=rng.choice(kinds),
                ids=ids, add=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)

    def even(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        # a few tokens stand out, the others fall off like a power of their rank: another power in each row
        power = 1.1 + 1.1 * even(B, 1)
        x = -power * torch.log(even(B, V) * V + 1e-3) + 0.3 * torch.randn((B, V), generator=g, device=dev)
        s["logits"] = (x + 8).to(getattr(torch, case["dtype"]))
        s["u"] = even(B)
        if case["temp"] == "one":
            s["temperature"] = torch.full((B,), 0.8, device=dev)
        else:  # each request its own, one of eight greedy
            s["temperature"] = torch.where(even(B) < 0.125, torch.zeros(B, device=dev), 0.6 + 0.8 * even(B))
        # 0 and 1: the call has no such filter; negative: each request its own, or none
        k, p, m = case["k"], case["p"], case["m"]
        some = lambda on, off: torch.where(even(B) < 0.7, on, torch.full_like(on, off))  # noqa: E731
        s["top_k"] = None if k == 0 else some((1 + 99 * even(B)).int(), 0) if k < 0 else torch.full(
            (B,), k, dtype=torch.int32, device=dev)
        s["top_p"] = None if p == 1 else some(0.7 + 0.29 * even(B), 1.0) if p < 0 else torch.full((B,), p, device=dev)
        s["min_p"] = None if m == 0 else some(0.01 + 0.1 * even(B), 0.0) if m < 0 else torch.full((B,), m, device=dev)
        return s
    n, rows, dim, streams = case["n"], case["rows"], case["dim"], case["streams"]
    if case["ids"] == "zipf":  # the r-th most frequent id in proportion to r ** -1.1
        ids = ((even(n) * (rows ** -0.1 - 1) + 1) ** -10 - 1).long().clamp(0, rows - 1)
        ids = ids * 7919 % rows
    else:
        ids = torch.randint(0, rows, (n,), generator=g, device=dev)
    s["pad"] = -1
    if case["ids"] == "padded":  # sequences end early
        s["pad"] = 0
        ids = torch.where(even(n) < 0.3, torch.zeros_like(ids), ids)
    s["ids"] = ids.to(torch.int32)
    s["scale"] = dim ** 0.5  # what a table of unit-length rows is looked up with
    kind = getattr(torch, case["table"])
    if case["op"] == "embed":
        table = torch.empty((rows, dim), dtype=kind, device=dev)
        s["table"] = table.normal_(0.0, dim ** -0.5, generator=g)
    else:
        s["dout"] = torch.randn((n, streams, dim), generator=g, device=dev).mul_(0.1).to(getattr(torch, case["grad"]))
        s["dtable"] = torch.empty((rows, dim), dtype=kind, device=dev)
        if case["add"]:
            s["dtable"].normal_(0.0, 1.0, generator=g)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return {"sample": _own_sample, "embed": _own_embed, "grad": _own_grad}[s["op"]](s)
    return {"sample": _plain_sample, "embed": _plain_embed, "grad": _plain_grad}[s["op"]](s)


def _plain_sample(s):
    x = s["logits"].double()  # 64 bits: sums over the vocabulary are compared with random numbers
    B, V = x.shape
    top = x.amax(1, keepdim=True)
    t = s["temperature"].double()[:, None]
    at = torch.arange(V, device=x.device)
    first = torch.where(x == top, at, V).amin(1, keepdim=True)
    w = torch.where(t == 0, (at == first).double(), torch.exp((x - top) / torch.where(t == 0, 1.0, t)))
    if s["top_k"] is not None or s["top_p"] is not None or s["min_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True)[1]
        ws = torch.gather(w, 1, order)
        stay = torch.ones_like(ws, dtype=torch.bool)
        if s["top_k"] is not None:
            k = s["top_k"][:, None]
            stay = (at < k) | (k <= 0)
            ws = torch.where(stay, ws, 0.0)
        if s["top_p"] is not None:
            p = s["top_p"].double()[:, None]
            upto = torch.cumsum(ws, 1)
            before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
            stay = stay & ((before < p * upto[:, -1:]) | (p >= 1))
        if s["min_p"] is not None:
            stay = stay & (ws >= s["min_p"].double()[:, None])
        stay[:, 0] = True
        kept = torch.zeros_like(stay).scatter_(1, order, stay)
        w = torch.where(kept, w, 0.0)
    cum = torch.cumsum(w, 1)
    total = cum[:, -1:]
    token = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    logprob = torch.log(torch.gather(w, 1, token) / total)
    return {"tokens": token[:, 0].to(torch.int32), "logprobs": logprob[:, 0].float()}


def _plain_embed(s):
    rows = (s["table"][s["ids"].long()].float() * s["scale"]).to(getattr(torch, s["out"]))
    return rows[:, None, :].expand(-1, s["streams"], -1).contiguous()


def _plain_grad(s):
    d = s["dout"].float().sum(1) * s["scale"]
    if s["pad"] >= 0:
        d = torch.where((s["ids"] == s["pad"])[:, None], 0.0, d)
    dt = s["dtable"]
    total = dt.float() if s["add"] else torch.zeros(dt.shape, dtype=torch.float32, device=dt.device)
    total.index_add_(0, s["ids"], d)  # (in place where the gradient that is there is fp32)
    return total if total.dtype == dt.dtype else dt.copy_(total)


def _kept(s, make):
    """What a program makes once and keeps: output and scratch buffers."""
    if "kept" not in s:
        import gram_memory_layer_amd as ge
        s["kept"] = (ge,) + make(ge)
    return s["kept"]


def _own_sample(s):
    def make(ge):
        B, V = s["logits"].shape
        dev = s["logits"].device
        size = ge.engram_sample_scratch_size(B, V)
        return (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.float32, device=dev),
                torch.empty(max(size, 1), dtype=torch.uint8, device=dev))
    ge, tokens, logprobs, scratch = _kept(s, make)
    ge.engram_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], tokens=tokens, logprobs=logprobs, scratch=scratch)
    return {"tokens": tokens, "logprobs": logprobs}


def _own_embed(s):
    def make(ge):
        shape = (s["n"], s["streams"], s["dim"])
        return (torch.empty(shape, dtype=getattr(torch, s["out"]), device=s["table"].device),)
    ge, out = _kept(s, make)
    return ge.engram_embed(s["table"], s["ids"], scale=s["scale"], streams=s["streams"], out=out)


def _own_grad(s):
    def make(ge):
        size = ge.engram_embed_grad_scratch_size(s["n"], s["rows"], s["dim"])
        return (torch.empty(max(size, 1), dtype=torch.uint8, device=s["dout"].device),)
    ge, scratch = _kept(s, make)
    return ge.engram_embed_grad(s["dout"], s["ids"], s["rows"], scale=s["scale"], pad_id=s["pad"],
                                dtable=s["dtable"], accumulate=s["add"], scratch=scratch)


# ------------------------------------------------------------------ the floor
_SIZE = {"float32": 4, "bfloat16": 2}


def _distinct(case):
    """How many rows the ids of a case are expected to name."""
    n, rows = case["n"], case["rows"]
    if case["ids"] != "zipf":
        return rows * (1 - (1 - 1 / rows) ** n)
    # whole ranks up to 4096, then ranks in steps of a tenth of themselves
    top = 1 - rows ** -0.1
    share = lambda a, b: (a ** -0.1 - min(b, rows) ** -0.1) / top  # noqa: E731
    found, r = 0.0, 1.0
    while r < rows:
        step = 1.0 if r < 4096 else min(r / 10, rows - r)
        found += step * (1 - (1 - share(r, r + step) / step) ** n)
        r += step
    return found


def work(case):
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": B * V * _SIZE[case["dtype"]] + B * 28, "flops": 4 * B * V}
    n, rows, dim, streams = case["n"], case["rows"], case["dim"], case["streams"]
    named = _distinct(case)
    if case["op"] == "embed":
        return {"bytes": 4 * n + named * dim * _SIZE[case["table"]] + n * streams * dim * _SIZE[case["out"]],
                "flops": n * dim}
    table = (2 * named if case["add"] else rows) * dim * _SIZE[case["table"]]
    return {"bytes": 4 * n + n * streams * dim * _SIZE[case["grad"]] + table, "flops": n * streams * dim}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        logprobs = []
        for b in range(case["B"]):
            x = s["logits"][b].double()
            t, u = float(s["temperature"][b]), float(s["u"][b])
            if t == 0:
                logprobs.append(0.0)
                continue
            values, order = torch.sort(x, descending=True, stable=True)
            k = int(s["top_k"][b]) if s["top_k"] is not None else 0
            n = min(k, x.numel()) if k > 0 else x.numel()
            prob = torch.softmax(values[:n] / t, 0)
            p = float(s["top_p"][b]) if s["top_p"] is not None else 1.0
            if p < 1:
                n = max(1, 1 + int((torch.cumsum(prob, 0)[:-1] < p).sum()))
            m = float(s["min_p"][b]) if s["min_p"] is not None else 0.0
            if m > 0:
                n = max(1, min(n, int((prob >= m * prob[0]).sum())))
            by_place, place = torch.sort(order[:n])
            prob = torch.softmax(values[:n] / t, 0)[place]
            pick = int(torch.searchsorted(torch.cumsum(prob, 0), u, right=True).clamp(max=n - 1))
            logprobs.append(float(torch.log(prob[pick])))
        return {"tokens": None, "logprobs": torch.tensor(logprobs, dtype=torch.float64, device=s["u"].device)}
    ids = s["ids"].long()
    if case["op"] == "embed":
        each = torch.index_select(s["table"], 0, ids).double() * s["scale"]
        return torch.stack([each] * case["streams"], 1)
    total = s["dtable"].double() if case["add"] else torch.zeros(
        (case["rows"], case["dim"]), dtype=torch.float64, device=ids.device)
    live = torch.nonzero(ids != s["pad"])[:, 0]
    if live.numel():
        each = s["dout"][live].double().sum(1) * s["scale"]
        total.index_put_((ids[live],), each, accumulate=True)
    return total
