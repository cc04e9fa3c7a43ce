"""engram_norm_quant's e8m0 scales where a group's largest value lies at 448 times
a power of two: the code is that of the exact value.

eps puts the chosen group's maximum within a few fp32 steps of the border; the
reference is the formula in 64 bits (sums of at most 32,768 exact squares: 1e-12
of the value at most), and a maximum within 1e-12 of the border is left open."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def at_the_border(ge, x, r, w, first, last):
    """Each row's group [first, last) at the border, all rows' scales checked; how many came near."""
    near = 0
    h = x.double() + r.double()
    ms, top = (h * h).mean(1), (h * w.double()).abs()
    rows, dim = x.shape
    for row in range(rows):
        m = top[row, first:last].max().item()
        if m == 0:
            continue
        lim = 1.75 * 2.0 ** np.floor(np.log2(0.9 * m / ms[row].item() ** 0.5 / 1.75))
        at = (m / lim) ** 2 - ms[row].item()
        for step in (-2, -1, 0, 1, 2):
            eps = float(np.float32(at) + step * np.spacing(np.float32(at)))
            y = torch.nn.functional.pad(top / torch.sqrt(ms + eps)[:, None], (0, -dim % 32))
            y = torch.log2(y.reshape(rows, -1, 32).amax(2) / 448).cpu()
            sure = (y - y.round()).abs() > 1e-12
            want = torch.where(y == -np.inf, 0, torch.ceil(y) + 127).to(torch.uint8)
            group = first // 32
            near += int((y[row, group] - y[row, group].round()).abs() < 2.0 ** -21)
            codes, scales, _ = ge.engram_norm_quant(x, w, residual=r, eps=eps)
            assert torch.equal(scales.cpu()[sure], want[sure]), (row, step)
            for inplace in (0, 1):
                a, b = x.clone(), r.clone()
                c2, s2, _ = ge.engram_norm_quant(a, w, residual=b, eps=eps, total=(a, b)[inplace])
                assert torch.equal(s2, scales) and torch.equal(c2, codes), (row, step, inplace)
    return near


@pytest.mark.parametrize("dim", [8, 40, 48, 56, 1032, 2064, 4120, 20504])
def test_a_short_last_group(ge, dim):
    """h is whole numbers: their squares' sum is exact in 32 bits too."""
    dev = torch.device("cuda:0")
    say("norm step, short group", dim)
    g = torch.Generator(device=dev)
    g.manual_seed(dim + 1)
    whole = lambda: torch.randint(-6, 7, (16, dim), generator=g, device=dev).bfloat16()  # noqa: E731
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=dev)).bfloat16()
    assert at_the_border(ge, whole(), whole(), w, dim // 32 * 32, dim) > 30


@pytest.mark.parametrize("dim", [32, 264, 1032, 5120, 32768])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** 20], ids=["even", "apart"])
def test_any_row(ge, dim, spread):
    """Squares whose sum 32 bits do not hold, and x and residual far `apart`, whose
    sum they do not hold either."""
    dev = torch.device("cuda:0")
    say("norm step, any values", dim, spread)
    g = torch.Generator(device=dev)
    g.manual_seed(dim + 2)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    x, res, w = r(64, dim).bfloat16(), (r(64, dim) / spread).bfloat16(), (1 + 0.1 * r(dim)).bfloat16()
    assert at_the_border(ge, x, res, w, 0, 32) > 100
