"""engram_sample where a cut falls among logits that weigh little each and much together,
and on scratch that held other numbers.

The header promises sums to 1e-11 of the row's.  So a cut is the formula's for a border moved
by at most that, and the token the formula's for a number moved by at most that, too: both
rise with them, so the token lies between those of both moved down and both moved up.  The
reference takes whole numbers of logits times weights in 80 bits (2^-63, times 2^22 at most)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_sample import KINDS, ge  # noqa: F401

pytestmark = pytest.mark.gpu
SUMS = 1e-11


def tail(V, dtype, dev, logits):
    """One logit of 0, and of two values the others, the lower ones last, so that the last that stays is the
    cut's: the row, and which value is where."""
    which = np.repeat(np.array([1, 2], dtype=np.int8), (V // 2, V - V // 2))
    which[V // 3] = 0
    values = torch.tensor([0.0, *logits], dtype=KINDS[dtype], device=dev)
    assert values.tolist() == [0.0, *logits]  # (no rounding)
    return values[torch.from_numpy(which).to(dev).long()][None], which


def token(which, w, k, border, number, moved):
    """The formula's token by counts; moved: of all sums, added to the border and the number."""
    n1, n2 = int((which == 1).sum()), int((which == 2).sum())
    n2 = min(n2, k - 1 - n1) if k else n2
    total = w[0] + n1 * w[1] + n2 * w[2]
    stay = int(np.ceil((border * total + moved * total - w[0] - n1 * w[1]) / w[2]))
    assert 100 < stay < n2 - 100  # the cut lies in the second value
    second = which == 2
    second &= np.cumsum(second) <= stay
    upto = (np.cumsum(which == 0) * w[0] + np.cumsum(which == 1) * w[1] + np.cumsum(second) * w[2])
    at = int(np.searchsorted(upto, number * upto[-1] + moved * total, side="right"))
    at = min(at, int(np.flatnonzero((which < 2) | second)[-1]))
    return at, w[which[at]] / upto[-1]


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("V,logits", [(20011, (-20.5, -20.625)), (129280, (-24.125, -24.25)), (129280, (-20.5, -20.625)),
                                      (262144, (-20.5, -21.0)), (1 << 22, (-20.5, -20.625)),
                                      (1 << 22, (-26.0, -26.125))])
def test_a_cut_among_small_weights(ge, V, logits, dtype):  # noqa: F811
    dev = torch.device("cuda:0")
    x, which = tail(V, dtype, dev, logits)
    w = np.exp(np.array([0.0, *logits], dtype=np.longdouble))
    total = w[0] + (which == 1).sum() * w[1] + (which == 2).sum() * w[2]
    p = np.float32(1 - (which == 2).sum() / 2 * w[2] / total)
    f = lambda v, kind=torch.float32: torch.tensor([v], dtype=kind, device=dev)  # noqa: E731
    for k in (0, V - 5):
        for u in (np.float32(1 - 2.0 ** -24), np.float32(1 - 2.0 ** -22)):
            say("sample small weights", V, logits, dtype, k, u)
            got, lp = ge.engram_sample(x, f(float(u)), top_p=f(float(p)), top_k=f(k, torch.int32) if k else None)
            border, number = np.longdouble(p), np.longdouble(u)
            least, most = (token(which, w, k, border, number, s * np.longdouble(SUMS))[0] for s in (-1, 1))
            share = token(which, w, k, border, number, np.longdouble(0))[1]
            assert least <= int(got) <= most, (int(got), least, most)
            if which[int(got)] == which[least] == which[most]:
                want = float(np.log(share))
                assert abs(float(lp) - want) <= 2.0 ** -24 * abs(want) + 1e-10


@pytest.mark.parametrize("dtype", KINDS)
def test_what_scratch_held_decides_nothing(ge, dtype):  # noqa: F811
    """Blocks of 8192 logits that a mask leaves empty: what the second kernel reads of them (the largest logits of
    groups, scratch's last array) is written by the first, so that no work depends on what was there."""
    dev = torch.device("cuda:0")
    say("sample scratch", dtype)
    B, V = 3, 65000
    groups = B * 8 * (2048 if dtype == "f32" else 1024) // 4
    x = torch.full((B, V), -float("inf"), dtype=KINDS[dtype], device=dev)
    x[0, 30000:30100] = torch.arange(100, device=dev) / 64
    x[1, ::20000] = 1.0
    x[2, V - 9:] = -2.0
    full = lambda v, kind=torch.float32: torch.full((B,), v, dtype=kind, device=dev)  # noqa: E731
    size = ge.engram_sample_scratch_size(B, V)
    last = B * 8 * 2048
    for kw in (dict(top_p=full(0.9)), dict(top_k=full(7, torch.int32)), dict(min_p=full(0.3))):
        seen = []
        for held in (0x00, 0x7F, 0xFF):  # 0x7F7F7F7F: 3.4e38, above every logit
            scratch = torch.full((size,), held, dtype=torch.uint8, device=dev)
            seen.append(ge.engram_sample(x, full(0.7), scratch=scratch, **kw))
            found = scratch[size - last:].view(torch.float32)[:groups].view(B, 8, -1)
            dead = torch.ones(B, 8, dtype=torch.bool, device=dev)
            dead[0, 3] = dead[2, 7] = False
            dead[1, [0, 2, 4, 7]] = False
            assert (found[dead] == -float("inf")).all(), held
        for got in seen[1:]:
            assert torch.equal(got[0], seen[0][0]) and torch.equal(got[1], seen[0][1])
