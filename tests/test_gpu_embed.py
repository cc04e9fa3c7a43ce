"""engram_embed and engram_embed_grad against plain forms in 64 bits.

Lookup: scale * value is one rounding to fp32 (2^-24 of it), then one to out's
type (bf16: 2^-8), and so is the reference's product rounded twice: bit for bit.

Gradient: a row's sum of N values in fp32, in any order, is off by at most
(N - 1) * 2^-24 * sum |d| (to first order; 1.01 for the rest), the scale and the
addition are one more rounding, 2^-24 of the result, and a bf16 row one of 2^-8."""
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -149  # a subnormal's step


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def guarded(shape, dtype, dev, fill=7.0):
    """A tensor with 64 values before and behind it, and those."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128,), fill, dtype=dtype, device=dev)
    return buf[64:64 + n].view(shape), (buf[:64], buf[64 + n:])


def check_grad(got, dout, ids, rows, scale, pad=-1, old=None):
    """dtable against the formula in 64 bits."""
    dim = dout.shape[-1]
    d = dout.reshape(ids.numel(), -1, dim).double()
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < rows) & (flat != pad)
    total = torch.zeros(rows, dim, dtype=torch.float64, device=d.device)
    mass, count = torch.zeros_like(total), torch.zeros(rows, dtype=torch.float64, device=d.device)
    total.index_add_(0, flat[live], d[live].sum(1))
    mass.index_add_(0, flat[live], d[live].abs().sum(1))
    count.index_add_(0, flat[live], torch.full_like(flat[live], d.shape[1], dtype=torch.float64))
    want = total * scale + (old.double() if old is not None else 0)
    bound = 1.01 * (count[:, None] - 1).clamp(min=0) * U32 * mass * abs(scale)
    bound = bound + U32 * (want.abs() + bound) + TINY
    if got.dtype == torch.bfloat16:
        bound = bound + U16 * (want.abs() + bound)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), ((off - bound).max().item(), want.flatten()[(off - bound).argmax()].item())
    untouched = count == 0
    if old is not None:  # not touched: the same bits
        assert torch.equal(got[untouched], old[untouched])
    else:
        assert (got[untouched] == 0).all()


@pytest.mark.parametrize("tk", KINDS)
@pytest.mark.parametrize("ok", KINDS)
@pytest.mark.parametrize("n,rows,dim,streams", [(1, 1, 8, 1), (1, 5, 64, 4), (7, 3, 24, 8), (64, 1000, 5120, 4),
                                                (613, 97, 1032, 3), (4097, 50, 64, 2), (3, 4, 32768, 1)])
def test_lookup(ge, n, rows, dim, streams, tk, ok):
    dev = torch.device("cuda:0")
    say("embed", n, rows, dim, streams, tk, ok)
    g = gen(dev, n + dim)
    table = torch.randn(rows, dim, generator=g, device=dev).to(KINDS[tk])
    ids = torch.randint(0, rows, (n,), generator=g, device=dev, dtype=torch.int32)
    ids[n // 2] = rows - 1
    for scale in (1.0, -dim ** 0.5, 1e-3):
        out, edges = guarded((n, streams, dim), KINDS[ok], dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        assert ge.engram_embed(table, ids, scale=scale, streams=streams, out=out, err=err) is out
        f32 = torch.tensor(scale, dtype=torch.float32).item()
        want = (table[ids.long()].double() * f32).float()  # (53 bits hold the product: one rounding)
        want = want.to(KINDS[ok])[:, None].expand(n, streams, dim)
        assert torch.equal(out, want)
        assert int(err.item()) == 0 and all((e == 7).all() for e in edges)


def test_lookup_shapes_types_and_bad_ids(ge):
    dev = torch.device("cuda:0")
    say("embed shapes")
    table = torch.randn(10, 16, device=dev)
    ids = torch.tensor([[0, 9, -1], [10, 3, 2 ** 31 - 1]], dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = ge.engram_embed(table, ids, err=err)
    assert out.shape == (2, 3, 16) and out.dtype == torch.float32 and int(err.item()) == ge.ERRBIT_ROW
    ok = torch.tensor([[1, 1, 0], [0, 1, 0]], dtype=torch.bool, device=dev)
    assert torch.equal(out[ok], table[ids[ok].long()]) and (out[~ok] == 0).all()
    out = ge.engram_embed(table, ids, streams=4, dtype=torch.bfloat16)
    assert out.shape == (2, 3, 4, 16) and out.dtype == torch.bfloat16
    assert ge.engram_embed(table, ids[:0], streams=2).shape == (0, 3, 2, 16)
    table[3, 5], table[3, 6], table[9, 0] = float("nan"), float("inf"), -float("inf")
    for kind in KINDS.values():
        out = ge.engram_embed(table.to(kind), ids, scale=2.0)
        assert torch.isnan(out[1, 1, 5]) and out[1, 1, 6] == float("inf") and out[0, 1, 0] == -float("inf")
        assert torch.isfinite(out[0, 0]).all()


@pytest.mark.parametrize("dk", KINDS)
@pytest.mark.parametrize("tk", KINDS)
@pytest.mark.parametrize("n,rows,dim,streams", [
    (1, 1, 8, 1), (1, 7, 64, 4), (16, 1000, 256, 4), (63, 2, 8, 1), (64, 3, 16, 3), (65, 1, 24, 2), (1111, 4001, 1032, 1),
    (4095, 300, 64, 1), (4096, 5000, 8, 5), (4097, 70000, 64, 1), (9000, 2049, 520, 2), (30011, 1 << 20, 64, 1)])
def test_gradient(ge, n, rows, dim, streams, dk, tk):
    dev = torch.device("cuda:0")
    say("embed grad", n, rows, dim, streams, dk, tk)
    g = gen(dev, n + rows)
    dout = torch.randn(n, streams, dim, generator=g, device=dev).to(KINDS[dk])
    even = torch.randint(0, rows, (n,), generator=g, device=dev, dtype=torch.int32)
    same = torch.full_like(even, rows // 2)
    skew = torch.where(torch.rand(n, generator=g, device=dev) < 0.5, same, even)
    for ids in (even, same, skew, torch.sort(skew)[0], torch.arange(n, device=dev).flip(0).int() % rows):
        for add in (False, True):
            dt, edges = guarded((rows, dim), KINDS[tk], dev)
            old = None
            if add:
                dt.copy_(torch.randn(rows, dim, generator=g, device=dev))
                old = dt.clone()
            size = ge.engram_embed_grad_scratch_size(n, rows, dim)
            scratch = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device=dev)
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            got = ge.engram_embed_grad(dout, ids, rows, scale=0.37, dtable=dt, accumulate=add,
                                       scratch=scratch[:size], err=err)
            assert got is dt
            check_grad(dt, dout, ids, rows, torch.tensor(0.37, dtype=torch.float32).item(), old=old)
            assert int(err.item()) == 0 and all((e == 7).all() for e in edges)
            assert (scratch[size:] == 0xAB).all()
            again = ge.engram_embed_grad(dout, ids, rows, scale=0.37, dtable=None if not add else old.clone(),
                                         accumulate=add, dtype=KINDS[tk])
            assert torch.equal(again, dt)  # the same bits on every run


@pytest.mark.parametrize("n", [65, 300, 8192, 8193])
def test_large_gradients_are_zero_between_the_rows(ge, n):
    dev = torch.device("cuda:0")
    rows, dim = 70_001, 1024  # 287 MB
    say("embed grad large", n)
    g = gen(dev, n)
    ids = torch.randint(0, rows, (n,), generator=g, device=dev, dtype=torch.int32)
    ids[n // 2:] = ids[0]
    dout = torch.randn(n, dim, generator=g, device=dev)
    dt, edges = guarded((rows, dim), torch.float32, dev)
    dt.fill_(float("nan"))
    ge.engram_embed_grad(dout, ids, rows, dtable=dt)
    check_grad(dt, dout, ids, rows, 1.0)
    assert all((e == 7).all() for e in edges)


@pytest.mark.parametrize("n", [50, 5000])
def test_gradient_pads_bad_ids_and_shapes(ge, n):
    dev = torch.device("cuda:0")
    say("embed grad pads", n)
    g = gen(dev, n)
    rows, dim = 37, 40
    ids = torch.randint(-2, rows + 2, (n,), generator=g, device=dev, dtype=torch.int32)
    ids[3] = -2 ** 31
    ids[5] = 2 ** 31 - 1
    dout = torch.randn(n, dim, generator=g, device=dev)
    dout[(ids < 0) | (ids >= rows) | (ids == 11)] = float("nan")  # what adds nothing is not looked at
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    old = torch.randn(rows, dim, generator=g, device=dev)
    for add in (False, True):
        err.zero_()
        dt = old.clone()
        ge.engram_embed_grad(dout, ids, rows, pad_id=11, dtable=dt, accumulate=add, err=err)
        check_grad(dt, torch.nan_to_num(dout), ids, rows, 1.0, pad=11, old=old if add else None)
        assert int(err.item()) == ge.ERRBIT_ROW
    # only pads; a pad is no error
    err.zero_()
    pads = torch.full_like(ids, 36)
    assert (ge.engram_embed_grad(dout, pads, rows, pad_id=36, err=err) == 0).all() and int(err.item()) == 0
    # [B, T] ids, with streams and without
    ids = (ids.clamp(0, rows - 1)).view(2, -1)
    d3 = torch.randn(2, n // 2, 3, dim, generator=g, device=dev)
    check_grad(ge.engram_embed_grad(d3, ids, rows), d3, ids, rows, 1.0)
    check_grad(ge.engram_embed_grad(d3[:, :, 0].contiguous(), ids, rows), d3[:, :, 0], ids, rows, 1.0)
    # nothing at all
    none = ge.engram_embed_grad(d3[:0], ids[:0], rows)
    assert none.shape == (rows, dim) and (none == 0).all()
    dt = old.clone()
    assert torch.equal(ge.engram_embed_grad(d3[:0], ids[:0], rows, dtable=dt, accumulate=True), old)


def test_gradient_keeps_a_bad_value_in_its_row(ge):
    dev = torch.device("cuda:0")
    say("embed grad nan")
    n, rows, dim = 3000, 40, 64
    ids = torch.randint(0, rows, (n,), device=dev, dtype=torch.int32)
    dout = torch.ones(n, dim, device=dev)
    dout[1234, 7], dout[99, 8] = float("nan"), float("inf")
    got = ge.engram_embed_grad(dout, ids, rows)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[ids[1234].long(), 7] = bad[ids[99].long(), 8] = True
    assert torch.isnan(got[ids[1234].long(), 7]) and got[ids[99].long(), 8] == float("inf")
    assert torch.equal(got[~bad], torch.bincount(ids.long(), minlength=rows)[:, None].float().expand(rows, dim)[~bad])


def test_gradient_is_the_lookups(ge):
    """Against differences: the sum of w * out moves by the gradient along a direction
    (linear, so exactly; whole numbers, so without a rounding)."""
    dev = torch.device("cuda:0")
    say("embed grad differences")
    g = gen(dev, 5)
    rows, dim, streams = 23, 16, 3
    ids = torch.randint(0, rows, (4, 50), generator=g, device=dev, dtype=torch.int32)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device=dev).float()  # noqa: E731
    table, step, w = whole(rows, dim), whole(rows, dim), whole(4, 50, streams, dim)
    loss = lambda t: (w.double() * ge.engram_embed(t, ids, scale=2.0, streams=streams).double()).sum().item()  # noqa: E731
    grad = ge.engram_embed_grad(w, ids, rows, scale=2.0)
    assert loss(table + step) - loss(table) == (grad.double() * step.double()).sum().item()


def test_offsets_past_32_bits(ge):
    dev = torch.device("cuda:0")
    say("embed far rows")
    rows, dim = 1_100_003, 4096  # bf16: 9.0 GB, more than 2^32 values
    table = torch.zeros(rows, dim, dtype=torch.bfloat16, device=dev)
    at = torch.tensor([0, 1, 524287, 524288, 1048575, 1048577, rows - 1], device=dev)
    table[at] = torch.randn(7, dim, device=dev).to(torch.bfloat16)
    ids = at.int().repeat(3)
    out = ge.engram_embed(table, ids, streams=2)
    assert torch.equal(out, table[ids.long()][:, None].expand(-1, 2, -1))
    old = table[at].clone()
    dout = torch.randn(21, dim, device=dev)
    ge.engram_embed_grad(dout, ids, rows, dtable=table, accumulate=True)
    check_grad(table[at], dout, torch.arange(7, device=dev).repeat(3), 7, 1.0, old=old)
    assert (table[at + 1 - 2 * (at > 0).long()][[0, 2]] == table[[1, 524286]]).all()
    table.fill_(3.0)
    ge.engram_embed_grad(dout, ids, rows, dtable=table)
    check_grad(table[at], dout, torch.arange(7, device=dev).repeat(3), 7, 1.0)
    table[at] = 0
    assert int(torch.count_nonzero(table.view(torch.int64))) == 0
    del table
    torch.cuda.empty_cache()


def test_many_positions(ge):
    """More chunks than one workgroup adds up; 4.8 GB of dout, past 2^31 values."""
    dev = torch.device("cuda:0")
    n, rows, dim = 300_007, 90_001, 8000
    say("embed grad many positions")
    g = gen(dev, 3)
    ids = torch.randint(0, rows, (n,), generator=g, device=dev, dtype=torch.int32)
    ids[torch.rand(n, generator=g, device=dev) < 0.1] = 77
    dout = torch.randint(-8, 9, (n, dim), generator=g, device=dev, dtype=torch.int8).to(torch.bfloat16)
    got = ge.engram_embed_grad(dout, ids, rows)
    # whole numbers below 2^24: exact in any order
    want = torch.zeros(rows, dim, device=dev)
    for i in range(0, n, 50_000):
        want.index_add_(0, ids[i:i + 50_000].long(), dout[i:i + 50_000].float())
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [62 * 2048, 62 * 2048 + 1, 8193, 5000])
def test_rows_named_by_most_positions(ge, n):
    """Whole numbers, summed exactly in any order: one row that every position, or most, names
    (counts that fill a sort's words; rows of one part to thousands), between rows named once."""
    dev = torch.device("cuda:0")
    g = gen(dev, n)
    for rows, dim in ((1, 72), (2, 8), (6, 8), (9, 64), (30, 8), (100, 136), (1000, 8), (40000, 64)):
        say(f"{n} positions of {rows} rows of {dim}")
        hot = rows // 2
        for share in (0.0, 0.02, 0.5):  # of positions that name another row
            ids = torch.where(torch.rand(n, generator=g, device=dev) < share,
                              torch.randint(0, rows, (n,), generator=g, device=dev), hot).int()
            dout = torch.randint(-3, 9, (n, dim), generator=g, device=dev).float()
            dt = ge.engram_embed_grad(dout, ids, rows)
            rest = ids != hot
            want = torch.zeros(rows, dim, dtype=torch.float64, device=dev)
            want.index_add_(0, ids[rest].long(), dout[rest].double())
            want[hot] = dout[~rest].double().sum(0)
            assert torch.equal(dt.double(), want), (rows, share)


def test_streams_of_work_and_graphs(ge):
    dev = torch.device("cuda:0")
    say("embed in a graph")
    g = gen(dev, 9)
    n, rows, dim, streams = 6000, 500, 64, 4
    table = torch.randn(rows, dim, generator=g, device=dev)
    ids = torch.randint(0, rows, (n,), generator=g, device=dev, dtype=torch.int32)
    dout = torch.randn(n, streams, dim, generator=g, device=dev)
    out = torch.empty(n, streams, dim, dtype=torch.bfloat16, device=dev)
    dt, acc = torch.empty(rows, dim, device=dev), torch.zeros(rows, dim, device=dev)
    scratch = torch.empty(ge.engram_embed_grad_scratch_size(n, rows, dim), dtype=torch.uint8, device=dev)

    def step():
        ge.engram_embed(table, ids, scale=3.0, streams=streams, out=out)
        ge.engram_embed_grad(dout, ids, rows, dtable=dt, scratch=scratch)
        ge.engram_embed_grad(dout, ids, rows, dtable=acc, accumulate=True, scratch=scratch)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    check_grad(dt, dout, ids, rows, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        ids.copy_(torch.roll(ids, 17))
        dout.mul_(0.5)
        acc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ge.engram_embed(table, ids, scale=3.0, streams=streams, dtype=torch.bfloat16)), r
        want = ge.engram_embed_grad(dout, ids, rows)
        assert torch.equal(dt, want) and torch.equal(acc, want), r
        check_grad(dt, dout, ids, rows, 1.0)


def test_refusals(ge):
    dev = torch.device("cuda:0")
    table = torch.zeros(10, 16, device=dev)
    ids = torch.zeros(4, dtype=torch.int32, device=dev)
    dout = torch.zeros(4, 16, device=dev)
    for call in (lambda: ge.engram_embed(table.half(), ids), lambda: ge.engram_embed(table, ids.long()),
                 lambda: ge.engram_embed(table, ids, dtype=torch.float16),
                 lambda: ge.engram_embed(table, ids, out=torch.empty(4, 16, device=dev), dtype=torch.bfloat16),
                 lambda: ge.engram_embed_grad(dout.half(), ids, 10),
                 lambda: ge.engram_embed_grad(dout, ids.long(), 10),
                 lambda: ge.engram_embed_grad(dout, ids, 10, dtable=table, dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ge.engram_embed(table.t(), ids), lambda: ge.engram_embed(table[0], ids),
                 lambda: ge.engram_embed(table, ids, out=torch.empty(5, 16, device=dev)),
                 lambda: ge.engram_embed(table.cpu(), ids),
                 lambda: ge.engram_embed_grad(dout[:3], ids, 10),
                 lambda: ge.engram_embed_grad(dout, ids, 11, dtable=table),
                 lambda: ge.engram_embed_grad(dout, ids, 10, accumulate=True)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ge.engram_embed(table, ids, scale=float("nan")),
                 lambda: ge.engram_embed(table, ids, streams=9),
                 lambda: ge.engram_embed(torch.zeros(4, 12, device=dev), ids),
                 lambda: ge.engram_embed_grad(dout, ids, 10, pad_id=10),
                 lambda: ge.engram_embed_grad(dout, ids, 10, scale=float("inf")),
                 lambda: ge.engram_embed_grad(dout, ids, 10, scratch=torch.empty(8, dtype=torch.uint8, device=dev))):
        with pytest.raises(ge.EngramError):
            call()
