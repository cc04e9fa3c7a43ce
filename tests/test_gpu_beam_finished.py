"""engram_beam_select with flags held as bool: the same bytes as in uint8."""
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_beam import check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ge():
    import gram_memory_layer_amd as ge
    ge.load()
    return ge


def test_bool_flags_in_place(ge):
    dev = torch.device("cuda:0")
    say("beam, bool flags")
    B, W, V = 5, 6, 3001
    x, c = draw(dev, B, W, V, torch.float32, 21)
    fin = torch.rand(B, W, generator=torch.Generator(device=dev).manual_seed(2), device=dev) < 0.3
    want = ge.engram_beam_select(x, c, finished=fin.to(torch.uint8), eos_id=7)
    check(want, x, c, fin, 7)
    for given in (fin.clone(), torch.ones_like(fin)):  # the input itself, and another tensor
        inout = given if torch.equal(given, fin) else fin.clone()
        got = ge.engram_beam_select(x, c, finished=inout, eos_id=7, new_finished=given)
        assert got[3] is given and given.dtype is torch.bool
        assert torch.equal(given.view(torch.uint8), want[3])
        assert all(torch.equal(p, q) for p, q in zip(got[:3], want[:3]))


def test_refused_flags(ge):
    dev = torch.device("cuda:0")
    x, c = draw(dev, 2, 3, 40, torch.float32, 1)
    with pytest.raises(TypeError):
        ge.engram_beam_select(x, c, new_finished=torch.zeros(2, 3, dtype=torch.int32, device=dev))
    for kind in (torch.bool, torch.uint8):
        with pytest.raises(ValueError):
            ge.engram_beam_select(x, c, new_finished=torch.zeros(2, 4, dtype=kind, device=dev))
        with pytest.raises(ValueError):
            ge.engram_beam_select(x, c, new_finished=torch.zeros(3, 2, dtype=kind, device=dev).t())
        with pytest.raises(ValueError):
            ge.engram_beam_select(x, c, new_finished=torch.zeros(2, 3, dtype=kind))
