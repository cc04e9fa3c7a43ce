"""engram_norm_quant against the formula in 64 bits.

h = x + r is formed in fp32 and total is its bf16 (both exactly those of
numpy's fp32 addition).  y in fp32 is off by at most d = (dim / 2 + 8) 2^-23 of
itself: the sum of squares by dim 2^-24 (all terms positive), halved by the
square root, the mean, eps, root and the two products by a few steps.  Then:
  code         |e4m3 * scale - y| <= 2^-4 |y| (1 + ...) + 2^-10 scale + d |y|
               (half a step of a normal; half the subnormal step 2^-9)
  e8m0 scale   the smallest power of two with max |y| <= 448 scale, for some
               max within (1 +- d) of the exact one
  fp32 scale   max |y| / 448 to d + 2^-23.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

FORMATS = ("e8m0_32", "f32_128", "f32_row")


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def check(x, r, w, eps, fmt, codes, scales, total):
    x32 = x.float().cpu().numpy().reshape(-1, x.shape[-1])
    h32 = x32 if r is None else x32 + r.float().cpu().numpy().reshape(x32.shape)
    if total is not None:
        want = torch.from_numpy(h32).to(torch.bfloat16)
        assert torch.equal(total.cpu().reshape(want.shape).view(torch.int16), want.view(torch.int16))
    rows, dim = h32.shape
    h = h32.astype(np.float64)
    ww = np.ones(dim) if w is None else w.double().cpu().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * ww
    d = (dim / 2 + 8) * 2.0 ** -23
    group = {"e8m0_32": 32, "f32_128": 128, "f32_row": dim}[fmt]
    ng = -(-dim // group)
    yp = np.zeros((rows, ng * group))
    yp[:, :dim] = np.abs(y)
    top = yp.reshape(rows, ng, group).max(2)
    s = scales.cpu().reshape(rows, ng)
    if fmt == "e8m0_32":
        c = s.numpy().astype(np.int64)
        scale = np.exp2(c - 127.0)
        assert (top * (1 - d) <= 448 * scale).all()
        assert ((c == 0) | (top * (1 + d) > 224 * scale)).all()
    else:
        scale = s.double().numpy()
        assert (np.abs(scale - top / 448) <= (d + 2.0 ** -23) * top / 448 + 2.0 ** -149).all()
    wide = np.repeat(scale, group, axis=1)[:, :dim]
    v = codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(rows, dim)
    assert np.isfinite(v).all()
    off = np.abs(v * wide - y)
    bound = 2.0 ** -4 * np.abs(y) * (1 + d) + 2.0 ** -10 * wide * (1 + 2.0 ** -20) + d * np.abs(y)
    bound += 448 * 2.0 ** -150  # a subnormal fp32 scale is off by half its step
    worst = (off / bound).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 16), (1, 32), (17, 40), (5, 128), (300, 136), (2, 256),
                                      (9, 1032), (4, 2056), (4, 5120), (33, 5120), (2, 16392), (1, 32768),
                                      (700, 520)])
def test_norm_quant(ge, fmt, rows, dim):
    dev = torch.device("cuda:0")
    say("norm", fmt, rows, dim)
    g = torch.Generator(device=dev)
    g.manual_seed(rows * 7 + dim)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    x, res, w = r(rows, dim, std=3.0), r(rows, dim), r(dim, std=0.2) + 1
    x[:, ::37] *= 50
    for residual in (None, res):
        for weight in (None, w):
            codes, scales, total = ge.engram_norm_quant(x, weight, residual=residual, scale_format=fmt)
            check(x, residual, weight, 1e-6, fmt, codes, scales, total)
            assert (total is None) == (residual is None)
    # any leading shape; bytes behind the last row stay
    buf = torch.full((rows + 1, dim), 77, dtype=torch.uint8, device=dev)
    c2, s2, _ = ge.engram_norm_quant(x.view(1, rows, dim), w, residual=res.view(1, rows, dim),
                                     scale_format=fmt, codes=buf[:rows].view(1, rows, dim))
    assert torch.equal(c2.view(rows, dim), codes) and torch.equal(s2.reshape(scales.shape), scales)
    assert (buf[rows] == 77).all()


def test_rows_past_32_bit_offsets(ge):
    dev = torch.device("cuda:0")
    say("norm far rows")
    rows, dim = 430000, 5120                               # 2.2e9 values
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device=dev)
    at = torch.tensor([0, 1, 209715, 209716, 419430, 419431, rows - 1], device=dev)
    x[at] = torch.randn(at.numel(), dim, device=dev).to(torch.bfloat16)
    codes, scales, total = ge.engram_norm_quant(x, residual=x, total=x)  # in place: total = 2 x
    few = (x[at].float() / 2).to(torch.bfloat16)
    check(few, few, None, 1e-6, "e8m0_32", codes[at], scales[at], x[at])
    assert (codes[2] == 0).all() and (codes[rows - 2] == 0).all()
    del x, codes, scales, total
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
def test_total_may_be_an_input(ge, fmt):
    dev = torch.device("cuda:0")
    say("norm in place", fmt)
    x = torch.randn(50, 1032, device=dev).to(torch.bfloat16)
    r = torch.randn(50, 1032, device=dev).to(torch.bfloat16)
    want = ge.engram_norm_quant(x, residual=r, scale_format=fmt)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        got = ge.engram_norm_quant(a, residual=b, scale_format=fmt, total=(a, b)[which])
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want))
        assert torch.equal((a, b)[1 - which], (x, r)[1 - which])
    one = x.clone()  # x twice
    got = ge.engram_norm_quant(one, residual=one, scale_format=fmt, total=one)
    check(x, x, None, 1e-6, fmt, *got)


@pytest.mark.parametrize("fmt", FORMATS)
def test_zeros_and_extremes(ge, fmt):
    dev = torch.device("cuda:0")
    say("norm extremes", fmt)
    x = torch.randn(6, 256, device=dev).to(torch.bfloat16)
    x[0] = 0                       # a row of zeros
    x[1, :128] = 0                 # groups of zeros
    x[2] *= 2.0 ** -60             # eps outweighs the mean of squares
    x[3] = 2.0 ** -133             # subnormals
    x[4] *= 2.0 ** 55
    x[5] = 1.0                     # all equal
    codes, scales, _ = ge.engram_norm_quant(x, scale_format=fmt)
    check(x, None, None, 1e-6, fmt, codes, scales, None)
    assert (codes[0] == 0).all() and (scales[0] == 0).all()
    # without eps a row of zeros is 0 * inf
    codes, _, _ = ge.engram_norm_quant(x[:1], scale_format=fmt, eps=0.0)
    assert (codes == 0x7F).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_and_infinity_stay_in_their_row(ge, fmt):
    dev = torch.device("cuda:0")
    say("norm NaN", fmt)
    x = torch.randn(5, 264, device=dev).to(torch.bfloat16)
    want = ge.engram_norm_quant(x, scale_format=fmt)
    y = x.clone()
    y[1, 7] = float("nan")
    y[3, 200] = float("-inf")
    codes, scales, _ = ge.engram_norm_quant(y, scale_format=fmt)
    for row in (0, 2, 4):
        assert torch.equal(codes[row], want[0][row]) and torch.equal(scales[row], want[1][row])
    assert (codes[1] == 0x7F).all()
    assert (scales[1] == 255).all() if fmt == "e8m0_32" else torch.isnan(scales[1]).all()
    rest = torch.arange(264, device=dev) != 200
    assert int(codes[3, 200]) == 0x7F and ((codes[3, rest] & 0x7F) == 0).all()  # finite / inf = 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_overflow_of_y_is_a_nan_code(ge, fmt):
    dev = torch.device("cuda:0")
    say("norm overflow", fmt)
    x = torch.ones(3, 256, device=dev, dtype=torch.bfloat16)
    x[:, 1::2] = -1.0
    x[1, 130] = 16.0                                       # y = 16 * rstd * 2^127 is past fp32
    w = torch.ones(256, device=dev, dtype=torch.bfloat16)
    w[130] = 2.0 ** 127
    codes, scales, _ = ge.engram_norm_quant(x, w, scale_format=fmt)
    assert int(codes[1, 130]) == 0x7F
    ok = torch.ones_like(codes, dtype=torch.bool)
    ok[1, 130] = False
    assert ((codes[ok] & 0x7F) != 0x7F).all()
    check(x[:, :128].contiguous(), None, None, 1e-6, fmt,
          *ge.engram_norm_quant(x[:, :128].contiguous(), scale_format=fmt))


def test_more_threads_than_a_launch_takes(ge):
    """2^26 + 13 short rows, in several launches: each as in a call of a few."""
    dev = torch.device("cuda:0")
    period, times = 17, 3947581
    say("norm launches", period * times)
    x = torch.randn(period, 8, device=dev, generator=torch.Generator(device=dev).manual_seed(5)).bfloat16()
    for fmt in ("e8m0_32", "f32_row"):
        few_codes, few_scales, _ = ge.engram_norm_quant(x, scale_format=fmt)
        codes = torch.full((period * times, 8), 0x7F, dtype=torch.uint8, device=dev)
        scales = torch.full((period * times, 1), 99, dtype=few_scales.dtype, device=dev)
        ge.engram_norm_quant(x.repeat(times, 1), scale_format=fmt, codes=codes, scales=scales)
        assert bool((codes.view(times, period, 8) == few_codes).all())
        assert bool((scales.view(times, period, 1) == few_scales).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_row_of_zeros_without_eps(ge, fmt):
    dev = torch.device("cuda:0")
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=dev)
    x[1] = 1
    codes, scales, _ = ge.engram_norm_quant(x, eps=0.0, scale_format=fmt)
    assert bool((codes[0] == 0x7F).all()) and bool((codes[1] != 0x7F).all())
    assert bool((scales[0] == 255).all() if fmt == "e8m0_32" else scales[0].isnan().all())


@pytest.mark.parametrize("dim", [64, 1032, 5120, 20488, 32768])
def test_a_step_of_the_scale_is_decided_in_64_bits(ge, dim):
    """eps puts a group's maximum within a few fp32 steps of 448 times a power of two.
    h is whole numbers, so that its squares' sum is exact; what is left is 64-bit
    rounding, 1e-12.  In place too."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(dim)
    rows, near = 32, 0
    whole = lambda: torch.randint(-6, 7, (rows, dim), generator=g, device=dev).bfloat16()  # noqa: E731
    x, r = whole(), whole()
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=dev)).bfloat16()
    h = x.double() + r.double()
    ms, top = (h * h).mean(1), (h * w.double()).abs()
    for row in range(rows):
        say("norm step", dim, row)
        m = top[row, :32].max().item()
        lim = 1.75 * 2.0 ** np.floor(np.log2(0.9 * m / ms[row].item() ** 0.5 / 1.75))
        at = (m / lim) ** 2 - ms[row].item()
        if at <= 0:
            continue
        for step in range(-3, 4):
            eps = float(np.float32(at) + step * np.spacing(np.float32(at)))
            y = torch.nn.functional.pad(top / torch.sqrt(ms + eps)[:, None], (0, -dim % 32))
            y = torch.log2(y.reshape(rows, -1, 32).amax(2) / 448).cpu()
            sure = (y - y.round()).abs() > 1e-12
            want = (torch.ceil(y) + 127).to(torch.uint8)
            near += int((y[row, 0] - y[row, 0].round()).abs() < 2.0 ** -21)
            codes, scales, _ = ge.engram_norm_quant(x, w, residual=r, eps=eps)
            assert torch.equal(scales.cpu()[sure], want[sure]), (row, step)
            for inplace in (0, 1):
                a, b = x.clone(), r.clone()
                c2, s2, _ = ge.engram_norm_quant(a, w, residual=b, eps=eps, total=(a, b)[inplace])
                assert torch.equal(s2, scales) and torch.equal(c2, codes), (row, step, inplace)
    assert near > 50


def test_refusals(ge):
    dev = torch.device("cuda:0")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        ge.engram_norm_quant(x.float())
    with pytest.raises(ValueError):
        ge.engram_norm_quant(x[:, ::2])
    with pytest.raises(ValueError):
        ge.engram_norm_quant(x, residual=x[:2])
    with pytest.raises(TypeError):
        ge.engram_norm_quant(x, scales=torch.empty(4, 2, device=dev))
    with pytest.raises(ge.EngramError) as e:
        ge.engram_norm_quant(torch.zeros(4, 12, dtype=torch.bfloat16, device=dev))
    assert e.value.status == 2
    codes, scales, total = ge.engram_norm_quant(x[:0], residual=x[:0])
    assert codes.shape == (0, 64) and scales.shape == (0, 2) and total.shape == (0, 64)
