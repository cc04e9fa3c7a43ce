"""engram_sample against a plain form in 64 bits.

Each weight is within 2e-12 of itself, so every sum of them is within 2e-12 of
itself, and roundings add less than 1e-11 of the total; the reference's own are
smaller.  So the token has to be the reference's, or one that the reference gives with
its top-p or its random number moved by 1e-10 of itself (a border that close is
rare, and none where the sums are whole numbers).  logprob is the fp32 nearest to a
value within 1e-10: off by 2^-24 of itself and 1e-10."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
NEAR = 1e-10
INF = float("inf")


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def one(x, u, t, k, p, m, moved_p=1.0, moved_u=1.0):
    """(token, logprob) of one row, x in float64."""
    V = x.size
    if not (0 <= t < INF and 0 <= p <= 1 and 0 <= m <= 1 and 0 <= u < 1):
        return -1, -INF
    if np.isnan(x).any() or (x == INF).any() or (x == -INF).all():
        return -1, -INF
    top = x.max()
    if t == 0:
        return int(np.argmax(x)), 0.0
    w = np.exp(np.maximum((x - top) / t, -1e4))
    w[(x == -INF) | (w < 2.0 ** -999)] = 0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -INF]
    if 1 <= k < V:
        order = order[:k]
    if p < 1:
        s = np.cumsum(w[order])
        before = np.concatenate([[0.0], s[:-1]])
        stay = before < p * moved_p * s[-1]
        stay[0] = True
        order = order[stay]
    if m > 0:
        order = order[w[order] >= m]
    kept = np.zeros(V)
    kept[order] = w[order]
    cum = np.cumsum(kept)
    token = int(np.searchsorted(cum, min(u * moved_u, 1 - 2.0 ** -30) * cum[-1], side="right"))
    return token, float(np.log(kept[token] / cum[-1]))


def check(ge, x, u, t=None, k=None, p=None, m=None, bits=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=x.device)
    tokens, logprobs = ge.engram_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m, err=err, **kw)
    assert int(err.item()) == bits
    B = x.shape[0]
    host = lambda v, off: [off] * B if v is None else v.double().cpu().tolist()  # noqa: E731
    xs = x.double().cpu().numpy()
    for b, (uu, tt, kk, pp, mm) in enumerate(zip(host(u, 0), host(t, 1), host(k, 0), host(p, 1), host(m, 0))):
        got, lp = int(tokens[b]), float(logprobs[b])
        want, wlp = one(xs[b], uu, tt, int(kk), pp, mm)
        if got != want:
            near = [one(xs[b], uu, tt, int(kk), pp, mm, 1 + s * NEAR, 1 + r * NEAR) for s in (-1, 0, 1) for r in (-1, 0, 1)]
            hit = [w for w in near if w[0] == got]
            assert hit, (b, got, want, uu, tt, kk, pp, mm)
            wlp = hit[0][1]
        assert lp == wlp or abs(lp - wlp) <= 2.0 ** -24 * abs(wlp) + NEAR, (b, lp, wlp, uu, tt, kk, pp, mm)
    return tokens, logprobs


def draw(dev, B, V, dtype, seed, ld=None, flat=False):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if flat:
        x = torch.randn(B, V, generator=g, device=dev) * 2
    else:  # falling like a power of the rank, another one in each row
        x = -(1.1 + 1.1 * torch.rand(B, 1, generator=g, device=dev)) * torch.log(
            torch.rand(B, V, generator=g, device=dev) * V + 1e-3)
    x = x.to(dtype)
    if ld is not None:
        wide = torch.full((B, ld), float("nan"), dtype=dtype, device=dev)
        wide[:, :V] = x
        x = wide[:, :V]
    return x, torch.rand(B, generator=g, device=dev), g


SIZES = [(1, 1), (1, 2), (3, 7), (2, 100), (5, 1000), (2, 8191), (2, 8192), (3, 8193), (4, 20011), (2, 32003), (3, 129280)]


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("B,V", SIZES)
@pytest.mark.parametrize("flat", [False, True])
def test_every_filter(ge, B, V, dtype, flat):
    dev = torch.device("cuda:0")
    say("sample", B, V, dtype, flat)
    x, u, g = draw(dev, B, V, KINDS[dtype], B * 7 + V, flat=flat)
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    check(ge, x, u)
    for t in (0.0, 0.3, 0.8, 1.0, 2.5):
        check(ge, x, u, t=full(t))
    for k in (1, 2, 40, 1000, V - 1, V, V + 5, -3, 5000, 20000):
        check(ge, x, u, t=full(0.8), k=full(k, torch.int32))
    for p in (0.0, 0.1, 0.5, 0.9, 0.99, 0.99999, 1.0):
        check(ge, x, u, t=full(0.8), p=full(p))
        check(ge, x, u, t=full(1.5), p=full(p), k=full(50, torch.int32))
        check(ge, x, u, p=full(p), k=full(V // 2, torch.int32))
    for m in (1e-30, 1e-5, 0.02, 0.3, 1.0):
        check(ge, x, u, m=full(m))
        check(ge, x, u, m=full(m), p=full(0.9))
        check(ge, x, u, t=full(0.7), m=full(m), k=full(30, torch.int32), p=full(0.95))
    # the ends of the random numbers
    for edge in (0.0, 1 - 2.0 ** -24):
        check(ge, x, full(edge))
        check(ge, x, full(edge), t=full(0.9), k=full(40, torch.int32), p=full(0.9), m=full(0.01))
        check(ge, x, full(edge), p=full(0.9))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("V", [50, 32003, 129280])
def test_a_batch_of_mixed_requests(ge, V, dtype):
    dev = torch.device("cuda:0")
    say("sample mixed", V, dtype)
    B = 64
    x, u, g = draw(dev, B, V, KINDS[dtype], V)
    r = lambda: torch.rand(B, generator=g, device=dev)  # noqa: E731
    t = torch.where(r() < 0.2, torch.zeros_like(u), 0.4 + r())
    k = torch.where(r() < 0.4, torch.zeros_like(u), 1 + 3000 * r() ** 4).int()
    p = torch.where(r() < 0.4, torch.ones_like(u), r())
    m = torch.where(r() < 0.5, torch.zeros_like(u), 0.3 * r() ** 3)
    first = check(ge, x, u, t, k, p, m)
    again = ge.engram_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    # a row's token does not depend on the rows beside it
    alone = ge.engram_sample(x[17:18], u[17:18], temperature=t[17:18], top_k=k[17:18], top_p=p[17:18], min_p=m[17:18])
    assert alone[0][0] == first[0][17] and alone[1][0] == first[1][17]


@pytest.mark.parametrize("ld,first", [(1001, 0), (1003, 1), (1024, 3), (4099, 5)])
@pytest.mark.parametrize("dtype", KINDS)
def test_rows_apart_and_at_any_element(ge, dtype, ld, first):
    dev = torch.device("cuda:0")
    say("sample rows", ld, first, dtype)
    B, V = 6, 997
    x, u, _ = draw(dev, B, V, KINDS[dtype], ld)
    buf = torch.full((B * ld + 16,), float("nan"), dtype=KINDS[dtype], device=dev)  # NaN between the rows
    rows = buf[first:first + B * ld].view(B, ld)[:, :V]
    rows.copy_(x)
    full = lambda v: torch.full((B,), v, device=dev)  # noqa: E731
    check(ge, rows, u)
    check(ge, rows, u, p=full(0.8))
    check(ge, rows, u, t=full(0.0))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("V", [4, 1000, 70000])
def test_ties(ge, dtype, V):
    """Equal logits: weights are 1 and sums whole numbers, so borders fall exactly."""
    dev = torch.device("cuda:0")
    say("sample ties", V, dtype)
    B = 8
    u = torch.arange(B, device=dev) / B
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    for value in (0.0, -7.5, 2.0 ** 100):
        x = torch.full((B, V), value, dtype=KINDS[dtype], device=dev)
        tokens, logprobs = check(ge, x, u)
        if V % B == 0:
            assert tokens.tolist() == [b * V // B for b in range(B)]
        check(ge, x, u, t=full(0.0))
        check(ge, x, u, p=full(0.5))
        check(ge, x, u, k=full(3, torch.int32))
        check(ge, x, u, k=full(max(1, V // 2), torch.int32), p=full(0.5))
        check(ge, x, u, m=full(1.0))
    # two levels: the upper one in a few places, the cut inside the lower one
    x = torch.zeros(B, V, dtype=KINDS[dtype], device=dev)
    x[:, V // 3::41] = 2.0
    n = x[0].count_nonzero().item()
    for k in (1, n, n + 1, n + 2, V - 1):
        check(ge, x, u, k=full(k, torch.int32))
    for p in (0.3, 0.6, 0.9):
        check(ge, x, u, p=full(p))
    x[:, 1::2] = -0.0  # both zeros are one
    check(ge, x, u, k=full(n + 3, torch.int32))
    check(ge, x, u, t=full(0.0))


@pytest.mark.parametrize("dtype", KINDS)
def test_masked_logits_and_bad_values(ge, dtype):
    dev = torch.device("cuda:0")
    say("sample masks", dtype)
    B, V = 8, 20000
    x, u, _ = draw(dev, B, V, KINDS[dtype], 3)
    x[0] = -INF                                         # nothing to choose
    x[1] = -INF
    x[1, 12345] = -3.0                                  # one token
    x[2] = torch.finfo(KINDS[dtype]).min                # masked by the type's lowest value
    x[2, 77] = 1.0
    x[3, 5:] = -INF                                     # fewer than top_k
    x[4] = torch.finfo(KINDS[dtype]).min                # nothing but the lowest value: all equal
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    for kw in (dict(), dict(t=full(0.0)), dict(k=full(50, torch.int32)), dict(p=full(0.9)), dict(m=full(0.1)),
               dict(k=full(50, torch.int32), p=full(0.9), m=full(0.01)), dict(p=full(0.99999), t=full(1.7)),
               dict(k=full(19999, torch.int32))):
        check(ge, x, u, **kw)
    x[5, V - 1] = float("nan")
    x[6, 0] = INF
    check(ge, x, u, bits=ge.ERRBIT_LOGIT)
    check(ge, x, u, t=full(0.0), bits=ge.ERRBIT_LOGIT)
    check(ge, x, u, k=full(9, torch.int32), p=full(0.5), bits=ge.ERRBIT_LOGIT)


@pytest.mark.parametrize("dtype", KINDS)
def test_bad_values_anywhere_without_a_filter(ge, dtype):
    dev = torch.device("cuda:0")
    V = 20000
    places = (0, 5, 1023, 2048, 3001, 8191, 8192, 12345, 16384, V - 1)
    for bad in (float("nan"), -float("nan"), INF):
        say("sample bad value", bad, dtype)
        x, u, _ = draw(dev, len(places) + 1, V, KINDS[dtype], 8)
        for b, v in enumerate(places):
            x[b, v] = bad
        check(ge, x, u, bits=ge.ERRBIT_LOGIT)
        check(ge, x, u, t=torch.full((len(places) + 1,), 0.7, device=dev), bits=ge.ERRBIT_LOGIT)
    x, u, _ = draw(dev, len(places), V, KINDS[dtype], 9)
    for b, v in enumerate(places):
        x[b, v] = -INF
        x[b, (v + 4000) % V] = torch.finfo(KINDS[dtype]).min
    check(ge, x, u)


def test_parameters_out_of_range(ge):
    dev = torch.device("cuda:0")
    say("sample parameters")
    x, u, _ = draw(dev, 6, 500, torch.float32, 2)
    row = lambda *v: torch.tensor(v, device=dev)  # noqa: E731
    nan = float("nan")
    bits = ge.ERRBIT_SAMPLE
    check(ge, x, row(0.5, 1.0, -0.1, nan, INF, 0.0), bits=bits)
    check(ge, x, u, t=row(1.0, -1.0, nan, INF, 0.0, 1e-30), bits=bits)
    check(ge, x, u, p=row(1.5, -0.1, nan, 0.5, 1.0, 0.0), bits=bits)
    check(ge, x, u, m=row(1.5, -0.1, nan, 0.5, 1.0, 0.0), bits=bits)
    x[1, 3] = nan
    check(ge, x, u, p=row(1.5, 0.1, 0.1, 0.5, 1.0, 0.0), bits=bits | ge.ERRBIT_LOGIT)


@pytest.mark.parametrize("dtype", KINDS)
def test_temperatures_and_spreads(ge, dtype):
    dev = torch.device("cuda:0")
    say("sample spread", dtype)
    B, V = 6, 30000
    x, u, _ = draw(dev, B, V, KINDS[dtype], 8, flat=True)
    x[0] *= 40
    x[1] *= 1e-3
    x[2] *= 1e-30
    if dtype == "f32":
        x[3] += 3e4
        x[4] *= 1e37
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    for t in (1e-38, 1e-6, 1.0, 30.0, 1e6, 3e38):
        check(ge, x, u, t=full(t))
        check(ge, x, u, t=full(t), p=full(0.7))
        check(ge, x, u, t=full(t), k=full(300, torch.int32), p=full(0.7))
        check(ge, x, u, t=full(t), m=full(0.05))


def test_the_draws_follow_the_distribution(ge):
    """Random numbers at the middles of 4096 equal steps: each token comes as often as
    its probability says, to one step."""
    dev = torch.device("cuda:0")
    say("sample distribution")
    V, n = 40, 4096
    x = torch.randn(1, V, device=dev).expand(n, V).contiguous()
    u = (torch.arange(n, device=dev) + 0.5) / n
    tokens, logprobs = ge.engram_sample(x, u)
    prob = torch.softmax(x[0].double(), 0)
    share = torch.bincount(tokens.long(), minlength=V).double() / n
    assert ((share - prob).abs() <= 1.0 / n).all()
    assert (tokens[1:] >= tokens[:-1]).all()
    assert (logprobs.double() - torch.log(prob)[tokens.long()]).abs().max() < 1e-6


def test_outputs_scratch_and_graphs(ge):
    dev = torch.device("cuda:0")
    say("sample in a graph")
    B, V = 9, 33333
    x, u, g = draw(dev, B, V, torch.float32, 12)
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    size = ge.engram_sample_scratch_size(B, V)
    buf = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device=dev)
    out = torch.full((B + 64,), 7, dtype=torch.int32, device=dev)
    lps = torch.full((B + 64,), 7.0, device=dev)
    kw = dict(temperature=full(0.9), top_k=full(0, torch.int32), top_p=full(0.95), min_p=full(0.001),
              tokens=out[:B], logprobs=lps[:B], scratch=buf[:size])
    graph = torch.cuda.CUDAGraph()
    kw["top_k"][::2] = 60
    kw["top_p"][::3] = 1.0
    kw["min_p"][:5] = 0.0
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ge.engram_sample(x, u, **kw)
    for r in range(3):
        x.copy_(torch.roll(x, 17, 1))
        u.copy_(torch.rand(B, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = check(ge, x, u, kw["temperature"], kw["top_k"], kw["top_p"], kw["min_p"])
        assert torch.equal(out[:B], want[0]) and torch.equal(lps[:B], want[1]), r
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ge.engram_sample(x, u, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    assert (buf[size:] == 0xAB).all() and (out[B:] == 7).all() and (lps[B:] == 7).all()
    # two calls at once, a scratch each
    x2, u2, _ = draw(dev, B, V, torch.bfloat16, 13)
    with torch.cuda.stream(side):
        a = [ge.engram_sample(x, u, temperature=kw["temperature"], top_p=kw["top_p"]) for _ in range(5)]
    b = [ge.engram_sample(x2, u2) for _ in range(5)]
    torch.cuda.synchronize()
    check(ge, x2, u2)
    assert all(torch.equal(r[0], a[0][0]) for r in a) and all(torch.equal(r[0], b[0][0]) for r in b)


def test_rows_past_32_bit_offsets(ge):
    dev = torch.device("cuda:0")
    say("sample far rows")
    B, V, ld = 5, 1111, 600_000_001
    buf = torch.empty((B - 1) * ld + V + 8, dtype=torch.bfloat16, device=dev)  # 4.8 GB
    rows = torch.as_strided(buf, (B, V), (ld, 1))
    x, u, _ = draw(dev, B, V, torch.bfloat16, 6)
    rows.copy_(x)
    check(ge, rows, u, p=torch.full((B,), 0.9, device=dev))
    check(ge, rows, u)
    del buf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", KINDS)
def test_the_largest_vocabulary(ge, dtype):
    dev = torch.device("cuda:0")
    V = 1 << 22
    say("sample largest", V)
    x, u, _ = draw(dev, 2, V, KINDS[dtype], 1, flat=True)
    full = lambda v, kind=torch.float32: torch.full((2,), v, dtype=kind, device=dev)  # noqa: E731
    check(ge, x, u)
    check(ge, x, u, p=full(0.9))
    check(ge, x, u, k=full(100, torch.int32))
    check(ge, x, u, k=full(1 << 21, torch.int32), p=full(0.9))


@pytest.mark.parametrize("dtype", KINDS)
def test_the_largest_vocabulary_behind_a_boundary(ge, dtype):
    """A row that begins inside 16 bytes reaches into one block more."""
    dev = torch.device("cuda:0")
    V, first = 1 << 22, 7 if dtype == "bf16" else 3
    say("sample largest vocabulary at element", first, dtype)
    buf = torch.full((V + 16,), -9.0, dtype=KINDS[dtype], device=dev)
    buf[first + V - 3:first + V] = 5.0
    x = buf[first:first + V][None]
    f = lambda v, kind=torch.float32: torch.tensor([v], dtype=kind, device=dev)  # noqa: E731
    for u in (0.0, 0.3, 0.7, 1 - 2.0 ** -24):
        check(ge, x, f(u))
        check(ge, x, f(u), k=f(2, torch.int32))
        check(ge, x, f(u), p=f(0.9))
        check(ge, x, f(u), k=f(4_000_000, torch.int32), p=f(0.99))
    buf.fill_(1.0)
    for u in (0.5, 1 - 2.0 ** -24):
        check(ge, x, f(u), p=f(0.75))
        check(ge, x, f(u), k=f(4_194_301, torch.int32))


def test_cuts_at_zeros_subnormals_and_the_ends_of_the_range(ge):
    dev = torch.device("cuda:0")
    tiny, huge = 2.0 ** -149, 3.0e38
    for V in (40, 900, 20011, 70001):
        g = torch.Generator(device=dev)
        g.manual_seed(V)
        for values in ((0.0, -0.0, tiny, -tiny), (0.0, -0.0), (-0.0, -1e-38, 1e-38, -tiny),
                       (0.0, -huge, -torch.finfo(torch.float32).max, -INF), (huge, -huge, 1.0, -INF)):
            say("sample zeros and ends", V, values)
            which = torch.randint(0, len(values), (3, V), generator=g, device=dev)
            x = torch.tensor(values, device=dev)[which]
            u = torch.rand(3, generator=g, device=dev)
            full = lambda v, kind=torch.float32: torch.full((3,), v, dtype=kind, device=dev)  # noqa: E731
            for k in (1, 7, V // 4, V // 3, V - 2):
                check(ge, x, u, k=full(k, torch.int32))
                check(ge, x, u, t=full(1e38), k=full(k, torch.int32), p=full(0.9))
            for p in (0.1, 0.5, 0.9):
                check(ge, x, u, p=full(p))
                check(ge, x, u, t=full(1e-40), p=full(p))
                check(ge, x, u, t=full(1e38), p=full(p), m=full(0.5))


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("values", [(1.0, 1.0078125, 0.99609375), (-2.0, -2.015625, -1.9921875), (0.0, -0.0, 2.0 ** -126)])
def test_more_logits_at_the_cut_than_the_list_holds(ge, dtype, values):
    """A few values, each many times: cuts among equal ones, top-p's among those that top-k cut."""
    dev = torch.device("cuda:0")
    for V in (30011, 129280):
        say("sample many equal", V, dtype, values)
        g = torch.Generator(device=dev)
        g.manual_seed(V)
        x = torch.tensor(values, device=dev)[torch.randint(0, 3, (4, V), generator=g, device=dev)].to(KINDS[dtype])
        x[1, ::5] = -INF
        x[2, ::7] = -5.0
        u = torch.rand(4, generator=g, device=dev)
        full = lambda v, kind=torch.float32: torch.full((4,), v, dtype=kind, device=dev)  # noqa: E731
        for p in (0.2, 0.5, 0.97):
            check(ge, x, u, p=full(p))
            check(ge, x, u, t=full(3.0), p=full(p), m=full(0.2))
        for k in (8193, 12345, V // 2, V - 5):
            check(ge, x, u, k=full(k, torch.int32))
            for p in (0.3, 0.9, 0.9999):
                check(ge, x, u, k=full(k, torch.int32), p=full(p))


def test_refusals(ge):
    dev = torch.device("cuda:0")
    x, u, _ = draw(dev, 3, 40, torch.float32, 1)
    for call in (lambda: ge.engram_sample(x.half(), u), lambda: ge.engram_sample(x, u.double()),
                 lambda: ge.engram_sample(x, u, top_k=u)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ge.engram_sample(x[0], u), lambda: ge.engram_sample(x, u[:2]),
                 lambda: ge.engram_sample(x.t().contiguous().t(), u), lambda: ge.engram_sample(x[:1].expand(3, 40), u),
                 lambda: ge.engram_sample(x, u.cpu()), lambda: ge.engram_sample(x, u, temperature=u[:2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ge.EngramError) as e:
        ge.engram_sample(x, u, scratch=torch.empty(8, dtype=torch.uint8, device=dev))
    assert e.value.status == 3
    assert all(t.shape == (0,) for t in ge.engram_sample(x[:0], u[:0]))
