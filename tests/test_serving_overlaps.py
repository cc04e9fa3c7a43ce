"""engram_beam_reorder refuses what it would read while it changes it (host checks
alone: nothing is launched)."""
import ctypes as C

import gram_memory_layer_amd as ge

FAKE = 1 << 20  # never dereferenced


def call(states, size, parents, B, W):
    p, s = (C.c_void_p * len(states))(*states), (C.c_int64 * len(size))(*size)
    return ge.load().engram_beam_reorder(p, s, len(states), parents, B, W, None, None)


def test_parents_among_the_states():
    # 2 * 4 rows of 8 bytes: 64 bytes; parents: 32 bytes
    assert call([FAKE], [8], FAKE, 2, 4) == 1
    assert call([FAKE], [8], FAKE + 60, 2, 4) == 1
    assert call([FAKE + 28], [8], FAKE, 2, 4) == 1
    assert call([FAKE + 4096, FAKE], [8, 8], FAKE + 4, 2, 4) == 1
    assert call([FAKE], [8], FAKE, 0, 4) == 0  # no sequences: nothing to do
