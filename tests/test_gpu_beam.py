"""engram_beam_select and engram_beam_reorder against plain forms in 64 bits.

The chosen tokens and parents have to be the reference's: its scores and the
library's (both 64-bit sums; the library's exponential to 1e-10) differ by less
than 1e-9, so two candidates may change places only where the reference has
them within 2e-9 of each other and not equal.  new_scores is the fp32 nearest
to a value within 1e-9: off by 2^-24 of itself and 1e-9."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu
NEAR = 2e-9


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def reference(logits, scores, finished, eos, pad):
    x = logits.double().cpu().numpy()
    c = scores.double().cpu().numpy()
    B, W = c.shape
    V = x.shape[-1]
    x = x.reshape(B, W, V)
    fin = np.zeros((B, W), bool) if finished is None else finished.cpu().numpy().astype(bool)
    score = np.full((B, W, V), -np.inf)
    for b in range(B):
        for w in range(W):
            if not np.isfinite(c[b, w]):
                continue
            if fin[b, w]:
                score[b, w, pad] = c[b, w]
                continue
            m = x[b, w].max()
            if np.isnan(m) or m == np.inf or m == -np.inf:
                continue
            d = x[b, w] - m  # first, or logits at the type's lowest value lose the rest
            score[b, w] = c[b, w] + (d - np.log(np.exp(d).sum()))
    flat = score.reshape(B, W * V)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :W + 1]
    best = np.take_along_axis(flat, order, 1)
    return flat, order, best, fin


def check(out, logits, scores, finished=None, eos=-1, pad=0):
    tokens, parents, new, done = (t.cpu().numpy() for t in out)
    flat, order, best, fin = reference(logits, scores, finished, eos, pad)
    B, W = tokens.shape
    V = flat.shape[1] // W
    for b in range(B):
        seen = set()
        for i in range(W):
            if best[b, i] == -np.inf:
                assert (tokens[b, i], parents[b, i], new[b, i], done[b, i]) == (pad, i, -np.inf, 0), (b, i)
                continue
            got = int(parents[b, i]) * V + int(tokens[b, i])
            assert 0 <= parents[b, i] < W and 0 <= tokens[b, i] < V and got not in seen, (b, i)
            seen.add(got)
            want = order[b, i]
            if got != want:  # only where the reference has them next to each other
                gap = abs(flat[b, got] - flat[b, want])
                assert 0 < gap <= NEAR, (b, i, got, want, flat[b, got], flat[b, want])
            assert abs(new[b, i] - flat[b, got]) <= 2.0 ** -24 * abs(flat[b, got]) + 1e-9, (b, i)
            assert done[b, i] == (fin[b, parents[b, i]] or tokens[b, i] == eos), (b, i)


def draw(dev, B, W, V, dtype, seed, ld=None):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn(B, 1, V, generator=g, device=dev) * 2 + 0.7 * torch.randn(B, W, V, generator=g, device=dev)
    x = x.to(dtype).reshape(B * W, V)
    if ld is not None:
        wide = torch.full((B * W, ld), float("nan"), dtype=dtype, device=dev)
        wide[:, :V] = x
        x = wide[:, :V]
    c = -torch.sort(torch.rand(B, W, generator=g, device=dev) * 8, dim=1)[0]
    return x, c


CASES = [(1, 1, 1), (1, 1, 2), (1, 4, 5), (2, 3, 7), (4, 1, 100), (3, 5, 1000), (1, 2, 511), (2, 4, 513),
         (2, 32, 4097), (5, 8, 2049), (1, 17, 8191), (1, 4, 129280), (3, 16, 20011), (40, 8, 32003),
         (64, 4, 1000), (200, 7, 333), (64, 8, 20000), (1, 32, 40), (16, 32, 9000), (300, 1, 5000),
         (300, 8, 7001), (100, 8, 20011)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,W,V", CASES)
def test_selection(ge, B, W, V, dtype):
    dev = torch.device("cuda:0")
    say("beam", B, W, V, dtype)
    x, c = draw(dev, B, W, V, dtype, B + W + V)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = ge.engram_beam_select(x, c, err=err)
    check(out, x, c)
    assert int(err.item()) == 0
    fin = torch.rand(B, W, device=dev) < 0.3
    for f in (fin, torch.ones_like(fin)):
        out = ge.engram_beam_select(x.view(B, W, V), c, finished=f, eos_id=V // 2, pad_id=V - 1)
        check(out, x, c, f, V // 2, V - 1)
    again = ge.engram_beam_select(x, c, finished=f, eos_id=V // 2, pad_id=V - 1)
    assert all(torch.equal(p, q) for p, q in zip(out, again))


@pytest.mark.parametrize("ld,first", [(1001, 0), (1003, 1), (1024, 3), (4099, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rows_apart_and_at_any_element(ge, dtype, ld, first):
    dev = torch.device("cuda:0")
    say("beam rows", ld, first, dtype)
    B, W, V = 3, 4, 997
    x, c = draw(dev, B, W, V, dtype, ld)
    buf = torch.full((B * W * ld + 16,), float("nan"), dtype=dtype, device=dev)  # NaN between the rows
    rows = buf[first:first + B * W * ld].view(B * W, ld)[:, :V]
    rows.copy_(x)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    check(ge.engram_beam_select(rows, c, err=err), rows, c)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,W,V", [(2, 4, 300), (1, 32, 5000), (40, 8, 20000)])
def test_ties_go_to_the_lowest_index(ge, B, W, V, dtype):
    dev = torch.device("cuda:0")
    say("beam ties", B, W, V, dtype)
    x = torch.zeros(B * W, V, dtype=dtype, device=dev)
    c = torch.zeros(B, W, device=dev)
    tokens, parents, _, _ = ge.engram_beam_select(x, c)
    assert (parents == 0).all() and torch.equal(tokens.cpu(), torch.arange(W, dtype=torch.int32).expand(B, W))
    # two levels, the upper one in a few places of every beam
    at = torch.arange(V // 3, V, 41, device=dev)
    x[:, at] = 2.0
    out = ge.engram_beam_select(x, c)
    check(out, x, c)
    c[:, W // 2:] = 1.0  # the upper half of the beams ahead
    check(ge.engram_beam_select(x, c), x, c)


def test_masked_logits_dead_beams_and_bad_values(ge):
    dev = torch.device("cuda:0")
    say("beam masks")
    inf = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        B, W, V = 9, 4, 1500
        x, c = draw(dev, B, W, V, dtype, 3)
        x[0:4] = -inf                                   # sequence 0: nothing to choose
        x[4, :] = -inf                                  # a beam with nothing, and one with a single token
        x[5, :] = -inf
        x[5, 1234] = -3.0
        x[6:8] = -inf
        x[8:12] = torch.finfo(dtype).min                # masked by the type's lowest value
        x[8, 77] = 1.0
        x[12:16, 3:] = -inf                             # fewer tokens than beams: 12 in all
        c[4, 1:] = -inf                                 # the first step
        c[5, :] = -inf                                  # all dead
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        check(ge.engram_beam_select(x, c, err=err, pad_id=5), x, c, pad=5)
        assert int(err.item()) == 0
        x[24, 1499] = float("nan")                      # sequence 6: a NaN, a +inf
        x[25, 0] = inf
        c[7, 2] = float("nan")
        c[8, 0] = inf
        check(ge.engram_beam_select(x, c, err=err, pad_id=5), x, c, pad=5)
        assert int(err.item()) == ge.ERRBIT_LOGIT
        # the dead and the finished beams' logits are not looked at
        err.zero_()
        x2, c2 = draw(dev, 2, 3, 700, dtype, 4)
        c2[0, 1] = -inf
        x2[1] = float("nan")
        fin = torch.zeros(2, 3, dtype=torch.uint8, device=dev)
        fin[1, 2] = 1
        x2[5] = inf
        check(ge.engram_beam_select(x2, c2, finished=fin, err=err), x2, c2, fin)
        assert int(err.item()) == 0


def test_spread_and_peaked_logits(ge):
    dev = torch.device("cuda:0")
    say("beam spread")
    B, W, V = 6, 8, 30000
    x, c = draw(dev, B, W, V, torch.float32, 8)
    x[:8] *= 40            # almost all mass on one token
    x[8:16] *= 1e-3        # almost flat
    x[16:24] += 3e4        # far from zero
    x[24:32] -= 1e30
    c[4] = -1e4
    check(ge.engram_beam_select(x, c), x, c)


def test_outputs_may_be_inputs_and_graphs(ge):
    dev = torch.device("cuda:0")
    say("beam in place, in a graph")
    B, W, V = 5, 6, 3001
    x, c = draw(dev, B, W, V, torch.float32, 12)
    fin = (torch.rand(B, W, device=dev) < 0.2).to(torch.uint8)
    want = ge.engram_beam_select(x, c, finished=fin, eos_id=7)
    cc, ff = c.clone(), fin.clone()
    got = ge.engram_beam_select(x, cc, finished=ff, eos_id=7, new_scores=cc, new_finished=ff)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    state = torch.arange(B * W * 2, dtype=torch.int32, device=dev).view(B * W, 2)
    start = state.clone()
    scratch = torch.empty(ge.engram_beam_select_scratch_size(B, W, V), dtype=torch.uint8, device=dev)
    outs = [torch.empty_like(t) for t in want]
    kw = dict(tokens=outs[0], parents=outs[1], new_scores=outs[2], new_finished=outs[3], scratch=scratch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ge.engram_beam_select(x, c, finished=fin, eos_id=7, **kw)
        ge.engram_beam_reorder([state], outs[1])
    for r in range(3):
        x.copy_(torch.roll(x, 17, 1))
        state.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        want = ge.engram_beam_select(x, c, finished=fin, eos_id=7)
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), r
        rows = (torch.arange(B, device=dev)[:, None] * W + want[1]).reshape(-1).long()
        assert torch.equal(state, start[rows]), r


def test_rows_past_32_bit_offsets(ge):
    dev = torch.device("cuda:0")
    say("beam far rows")
    B, W, V, ld = 1, 5, 1111, 600_000_001
    buf = torch.empty(4 * ld + V + 8, dtype=torch.bfloat16, device=dev)  # 4.8 GB
    rows = torch.as_strided(buf, (W, V), (ld, 1))
    x, c = draw(dev, B, W, V, torch.bfloat16, 6)
    rows.copy_(x)
    check(ge.engram_beam_select(rows, c), rows, c)
    del buf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,W,V", [(2, 4, 300), (1, 2, 129280), (3, 5, 777), (1, 1, 1)])
def test_flat_rows_at_any_score(ge, B, W, V, dtype):
    """Rows of one value (a fresh head's zeros), where score and log sum cancel to
    rounding errors, also with scores beside which the logits vanish."""
    dev = torch.device("cuda:0")
    for value in (0.0, 1e-30, -5.0, 2.0 ** 100):
        x = torch.full((B * W, V), value, dtype=dtype, device=dev)
        for c0 in (0.0, -0.1, -3.7, -11.77, -1234.5, -1e6, -3e38, 1e30):
            say("beam flat", B, W, V, dtype, value, c0)
            same = torch.full((B, W), c0, device=dev)
            check(ge.engram_beam_select(x, same), x, same)
            apart = same - 0.37 * torch.arange(W, device=dev)
            check(ge.engram_beam_select(x, apart), x, apart)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1001, 32003])
def test_beams_of_the_same_logits_tie(ge, dtype, V):
    """Rows that start at different places of a 16-byte line, the same in each."""
    dev = torch.device("cuda:0")
    B, W = 4, 5
    say("beam same rows", V, dtype)
    x, _ = draw(dev, B, 1, V, dtype, V)
    x = x.view(B, 1, V).expand(B, W, V).reshape(B * W, V).contiguous()
    c = torch.full((B, W), -1.25, device=dev)
    check(ge.engram_beam_select(x, c), x, c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_nearly_flat_rows(ge, dtype):
    dev = torch.device("cuda:0")
    B, W, V = 2, 4, 5000
    for step in (2.0 ** -20, 2.0 ** -100):
        x = torch.zeros(B * W, V, dtype=dtype, device=dev)
        x[:, 4321], x[:, 17], x[:, 99] = step, 2 * step, -step
        c = -torch.rand(B, W, device=dev, generator=torch.Generator(device=dev).manual_seed(3)) - 1
        tokens, parents, new, _ = (t.cpu() for t in ge.engram_beam_select(x, c))
        best = c.argmax(1).cpu()
        assert torch.equal(parents, best[:, None].expand(B, W).int())
        if step == 2.0 ** -20:  # steps of 1e-6 show in a 64-bit score, 1e-30 is a tie
            assert tokens.tolist() == [[17, 4321, 0, 1]] * B
        else:
            assert tokens.tolist() == [[0, 1, 2, 3]] * B
        want = c.double().cpu().gather(1, best[:, None]) - np.log(V)
        assert ((new.double() - want).abs() <= 2.0 ** -24 * want.abs() + 1e-9 + 2 * step).all()


def test_selection_refusals(ge):
    dev = torch.device("cuda:0")
    x, c = draw(dev, 2, 3, 40, torch.float32, 1)
    with pytest.raises(TypeError):
        ge.engram_beam_select(x.half(), c)
    with pytest.raises(ValueError):
        ge.engram_beam_select(x[:5], c)
    with pytest.raises(ValueError):
        ge.engram_beam_select(x.t().contiguous().t(), c)
    with pytest.raises(ValueError):
        ge.engram_beam_select(x, c.reshape(-1))
    for kw in (dict(pad_id=40), dict(pad_id=-1), dict(eos_id=-5)):
        with pytest.raises(ge.EngramError):
            ge.engram_beam_select(x, c, **kw)
    with pytest.raises(ge.EngramError) as e:
        ge.engram_beam_select(x, c, scratch=torch.empty(8, dtype=torch.uint8, device=dev))
    assert e.value.status == 3
    out = ge.engram_beam_select(x[:0], c[:0])
    assert all(t.shape == (0, 3) for t in out)


@pytest.mark.parametrize("B,W", [(1, 1), (1, 2), (3, 3), (2, 4), (64, 8), (5, 16), (2, 17), (3, 32), (300, 5)])
def test_reorder(ge, B, W):
    dev = torch.device("cuda:0")
    say("reorder", B, W)
    g = torch.Generator(device=dev)
    g.manual_seed(B * 40 + W)
    parents = torch.randint(0, W, (B, W), generator=g, device=dev, dtype=torch.int32)
    rows = (torch.arange(B, device=dev)[:, None] * W + parents).reshape(-1).long()
    sets = [[(2,)], [(2,)] * 8, [(1,)], [(4,), (4,)], [(3,), (8,), (128,), (129,)], [(256, 4)], [(513,)], [(6000,), (2,)],
            [(4,)] * 32]
    for shapes in sets:
        for skew in (0, 1, 2):  # pointers at 16, 4 and 8 bytes
            base = []
            for s in shapes:
                n = B * W * int(np.prod(s))
                buf = torch.randint(-2 ** 31, 2 ** 31 - 1, (n + 8,), generator=g, device=dev, dtype=torch.int32)
                base.append((buf, buf[skew:skew + n].view(B * W, *s)))
            want = [st[rows].clone() for _, st in base]
            edge = [(buf[:skew].clone(), buf[skew + st.numel():].clone()) for buf, st in base]
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            ge.engram_beam_reorder([st for _, st in base], parents, err=err)
            assert all(torch.equal(st, x) for (_, st), x in zip(base, want)), (shapes, skew)
            for (buf, st), (lo, hi) in zip(base, edge):
                assert torch.equal(buf[:skew], lo) and torch.equal(buf[skew + st.numel():], hi)
            assert int(err.item()) == 0


def test_reorder_past_32_bit_offsets(ge):
    dev = torch.device("cuda:0")
    say("reorder far")
    B, W, words = 2, 4, 180_000_003                        # 5.8 GB in all
    st = torch.empty(B * W, words, dtype=torch.int32, device=dev)
    mark = torch.arange(B * W, device=dev, dtype=torch.int32)
    cols = torch.tensor([0, 1, 2, words // 2, words - 2, words - 1], device=dev)
    st[:, cols] = mark[:, None] * 100 + torch.arange(6, device=dev, dtype=torch.int32)
    before = st[:, cols].clone()
    parents = torch.tensor([[1, 1, 3, 0], [3, 0, 2, 2]], dtype=torch.int32, device=dev)
    ge.engram_beam_reorder([st], parents)
    rows = (torch.arange(B, device=dev)[:, None] * W + parents).reshape(-1).long()
    assert torch.equal(st[:, cols], before[rows])
    del st
    torch.cuda.empty_cache()


def test_reorder_of_more_threads_than_a_launch_takes(ge):
    """Rows of 2^31 + 4097 words: more than 2^23 workgroups, in several launches."""
    dev = torch.device("cuda:0")
    R = 2 ** 31 + 4097
    if torch.cuda.mem_get_info()[0] < 2.2 * 8 * R:
        pytest.skip("needs %d GB" % (8 * R >> 30))
    say("reorder launches", R)
    st = torch.zeros(2 * R + 1, dtype=torch.int32, device=dev)[1:].view(2, R)
    at = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 255, R - 257, R - 1], device=dev)
    st[0, at] = torch.arange(7, dtype=torch.int32, device=dev) + 1
    st[1, at] = torch.arange(7, dtype=torch.int32, device=dev) + 11
    ge.engram_beam_reorder([st], torch.tensor([[1, 0]], dtype=torch.int32, device=dev))
    assert st[0, at].tolist() == list(range(11, 18)) and st[1, at].tolist() == list(range(1, 8))
    ge.engram_beam_reorder([st], torch.tensor([[1, 1]], dtype=torch.int32, device=dev))
    assert st[0, at].tolist() == list(range(1, 8)) and st[1, at].tolist() == list(range(1, 8))


def test_reorder_types_bad_parents_and_refusals(ge):
    dev = torch.device("cuda:0")
    say("reorder types")
    B, W = 3, 4
    parents = torch.tensor([[3, 2, 1, 0], [0, 0, 0, 0], [1, 4, -1, 2]], dtype=torch.int32, device=dev)
    x = torch.randn(B, W, 6, device=dev).to(torch.bfloat16)
    y = torch.randint(0, 255, (B * W, 12), dtype=torch.uint8, device=dev)
    x0, y0 = x.clone(), y.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ge.engram_beam_reorder([x, y], parents, err=err)
    assert int(err.item()) == ge.ERRBIT_PARENT
    src = torch.tensor([[3, 2, 1, 0], [0, 0, 0, 0], [1, 1, 2, 2]], device=dev)
    rows = (torch.arange(B, device=dev)[:, None] * W + src).reshape(-1)
    assert torch.equal(x.view(B * W, 6), x0.view(B * W, 6)[rows]) and torch.equal(y, y0[rows])
    with pytest.raises(ge.EngramError):
        ge.engram_beam_reorder([x, x], parents)
    with pytest.raises(ge.EngramError):
        ge.engram_beam_reorder([y.view(-1)[:B * W * 6].view(B * W, 6)], parents)  # rows of 6 bytes
    with pytest.raises(ValueError):
        ge.engram_beam_reorder([x[:2]], parents)
    with pytest.raises(TypeError):
        ge.engram_beam_reorder([x], parents.long())
    assert ge.engram_beam_reorder([x[:0]], parents[:0])[0].numel() == 0
