"""engram_norm_quant's codes and scales against its formula operation by
operation: y = (h * rstd) * weight and y / scale in fp32, each rounded once.

What fp32 leaves open is rstd: a thread sums at most 32 squares in fp32 (each
addition off by at most 2^-24 of the sum, all terms positive), the rest is 64
bits, so the mean is within 32 * 2^-24 of the exact one, its root within 16 *
2^-24, which is at most 16 steps, and one more for rstd's own rounding.  Some
rstd within 17 steps of the exact one gives a row's codes and scales bit for
bit."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_norm_quant import FORMATS, check

pytestmark = pytest.mark.gpu
STEPS = 17


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def e4m3(v):
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def by_steps(h, w, rstd, fmt):
    """(codes, scales) of rows h in fp32, with one rstd a row."""
    rows, dim = h.shape
    y = (h * rstd[:, None]) * w
    group = {"e8m0_32": 32, "f32_128": 128, "f32_row": dim}[fmt]
    ng = -(-dim // group)
    top = np.zeros((rows, ng * group), np.float32)
    top[:, :dim] = np.abs(y)
    top = top.reshape(rows, ng, group).max(2)
    if fmt == "e8m0_32":
        m, e = np.frexp(top)
        code = np.where(top > 0, np.maximum(np.where(m > 0.875, e - 8, e - 9) + 127, 0), 0)
        wide = np.repeat(np.ldexp(np.float32(1), code - 127), group, axis=1)[:, :dim]
        return e4m3((y.astype(np.float64) / wide).astype(np.float32)), code.astype(np.uint8)
    scale = top / np.float32(448)
    wide = np.repeat(scale, group, axis=1)[:, :dim]
    return e4m3(np.where(wide > 0, y / np.where(wide > 0, wide, 1), 0).astype(np.float32)), scale


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,dim,residual", [(1111, 1032, False), (96, 5120, True), (300, 136, True), (8, 32768, False)])
def test_codes_are_the_formulas(ge, fmt, rows, dim, residual):
    dev = torch.device("cuda:0")
    say("norm by steps", fmt, rows, dim)
    g = torch.Generator(device=dev)
    g.manual_seed(rows + dim)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    x, res, w = r(rows, dim, std=2.0), r(rows, dim, std=0.5) if residual else None, r(dim, std=0.05) + 1
    x[:, 5] *= 24
    codes, scales, _ = ge.engram_norm_quant(x, w, residual=res, scale_format=fmt)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    h = x.float().cpu().numpy()
    if residual:
        h = h + res.float().cpu().numpy()
    exact = 1 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + float(np.float32(1e-6)))
    found = np.zeros(rows, bool)
    for k in sorted(range(-STEPS, STEPS + 1), key=abs):
        at = np.nonzero(~found)[0]
        if not at.size:
            break
        near = exact[at].astype(np.float32)
        c, s = by_steps(h[at], w.float().cpu().numpy(), near + np.float32(k) * np.spacing(near), fmt)
        found[at] = (c == codes[at]).all(1) & (s == scales[at]).all(1)
    assert found.all(), np.nonzero(~found)[0]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x0,w0,eps", [(2.0 ** 50, 2.0 ** 80, 1e-6),    # h * weight is past fp32, y is not
                                       (2.0 ** -60, 2.0 ** -60, 0.0),  # rstd over the scale is past it
                                       (2.0 ** -60, 2.0 ** -80, 0.0),  # h * weight is subnormal
                                       (2.0 ** -63, 2.0 ** 100, 0.0),
                                       (1.0, 2.0 ** 120, 1e-6)])
def test_only_y_has_to_fit(ge, fmt, x0, w0, eps):
    dev = torch.device("cuda:0")
    say("norm range", fmt, x0, w0)
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    x, w = r(5, 296) * x0, (r(296).abs() + 1) * w0
    codes, scales, _ = ge.engram_norm_quant(x, w, eps=eps, scale_format=fmt)
    check(x, None, w, eps, fmt, codes, scales, None)


@pytest.mark.parametrize("fmt", FORMATS[1:])
@pytest.mark.parametrize("e", range(-143, -130))
def test_subnormal_scales(ge, fmt, e):
    """A scale below fp32's normal numbers is a whole number of 2^-149: the codes go
    with the scale that is stored, a scale of zero has codes of zero.  y is off by
    2^-150, 448 scales by 448 times that, beside the code's own half step."""
    dev = torch.device("cuda:0")
    say("norm subnormal scale", fmt, e)
    g = torch.Generator(device=dev)
    g.manual_seed(e + 200)
    x = (torch.randn(40, 256, generator=g, device=dev) * 2.0 ** (e + 120)).to(torch.bfloat16)
    w = torch.full((256,), 2.0 ** -130, dtype=torch.bfloat16, device=dev)  # eps: rstd is near 2^10
    codes, scales, _ = ge.engram_norm_quant(x, w, scale_format=fmt)
    h = x.double().cpu().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * w.double().cpu().numpy()
    wide = scales.double().cpu().numpy().repeat(256 // scales.shape[1], axis=1)
    v = codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    assert np.isfinite(v).all()
    bound = 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -15) + 2.0 ** -10 * wide + 449 * 2.0 ** -150
    # half a code's step, and where the scale is short of most / 448 the cut at 448
    assert (np.abs(v * wide - y) <= bound).all()
    lo = np.abs(y) <= 440 * wide  # not cut: half a code's step alone
    near = 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -15) + 2.0 ** -10 * wide + 2.0 ** -149
    assert (np.abs(v * wide - y)[lo] <= near[lo]).all()
