"""The calls at the vocabulary's two ends (lookup, its gradient, sampling)
without a GPU: sizes and refusals.  Every call here fails its checks on the
host, or has no work, and launches nothing."""
import pytest
import torch

import gram_memory_layer_amd as ge

FAKE = 1 << 20  # never dereferenced


def test_embed_host_checks():
    lib = ge.load()

    def call(table=FAKE, t32=0, rows=100, dim=64, ids=FAKE, n=4, scale=1.0, streams=1, out=FAKE, o32=0):
        return lib.engram_embed(table, t32, rows, dim, ids, n, scale, streams, out, o32, None, None)
    assert call(table=None) == 1 and call(ids=None) == 1 and call(out=None) == 1
    assert call(table=FAKE + 8) == 1 and call(out=FAKE + 4) == 1 and call(ids=FAKE + 2) == 1
    assert call(t32=2) == 1 and call(o32=-1) == 1
    assert call(rows=0) == 1 and call(n=-1) == 1 and call(n=1 << 31) == 1 and call(streams=0) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(rows=1 << 31) == 2 and call(streams=9) == 2
    for dim in (0, 4, 12, 32776):
        assert call(dim=dim) == 2, dim
    assert call(n=0) == 0 and call(n=0, table=None, ids=None, out=None) == 0


def test_embed_grad_host_checks():
    lib = ge.load()
    size = ge.engram_embed_grad_scratch_size
    assert size(0, 100, 64) == 0 and size(-1, 100, 64) == 0 and size(4, 0, 64) == 0 and size(4, 100, 12) == 0
    assert 0 < size(4, 100, 64) <= size(4096, 100, 64) < size(4097, 100, 64)
    assert size((1 << 31) - 1, 100, 32768) == 0  # more tiles than a launch takes

    def call(dout=FAKE, d32=0, ids=FAKE, n=4, streams=1, rows=100, dim=64, scale=1.0, pad=-1, add=0, dt=FAKE,
             t32=0, scratch=FAKE, nbytes=1 << 30):
        return lib.engram_embed_grad(dout, d32, ids, n, streams, rows, dim, scale, pad, add, dt, t32, scratch,
                                     nbytes, None, None)
    assert call(dout=None) == 1 and call(ids=None) == 1 and call(dt=None) == 1
    assert call(dout=FAKE + 8) == 1 and call(dt=FAKE + 4) == 1 and call(ids=FAKE + 2) == 1
    assert call(d32=2) == 1 and call(t32=2) == 1 and call(add=2) == 1
    assert call(n=-1) == 1 and call(rows=0) == 1 and call(streams=0) == 1
    assert call(pad=-2) == 1 and call(pad=100) == 1
    assert call(scale=float("nan")) == 1 and call(scale=-float("inf")) == 1
    assert call(rows=1 << 31) == 2 and call(streams=9) == 2 and call(dim=12) == 2
    assert call(n=(1 << 31) - 1, dim=32768) == 2
    assert call(scratch=None) == 3 and call(scratch=FAKE + 128) == 3
    assert call(nbytes=size(4, 100, 64) - 1) == 3
    assert call(n=0, add=1) == 0 and call(n=0, add=0, dt=None) == 1


def test_binding_refuses_what_is_not_on_the_device():
    table, ids = torch.zeros(10, 16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ge.engram_embed(table, ids)
    with pytest.raises(TypeError):
        ge.engram_embed(table.double(), ids)
    with pytest.raises(TypeError):
        ge.engram_embed([1.0], ids)
    with pytest.raises(ValueError):
        ge.engram_embed_grad(torch.zeros(4, 16), ids, 10)


def test_sample_host_checks():
    lib = ge.load()
    size = ge.engram_sample_scratch_size
    assert size(2, 1000) > 0 and size(0, 1000) == 0 and size(2, 0) == 0 and size(2, (1 << 22) + 1) == 0

    def call(logits=FAKE, f32=1, ld=1000, u=FAKE, t=None, k=None, p=None, m=None, B=2, V=1000, tok=FAKE, lp=None,
             scratch=FAKE, nbytes=1 << 40):
        return lib.engram_sample(logits, f32, ld, u, t, k, p, m, B, V, tok, lp, scratch, nbytes, None, None)
    assert call(logits=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(logits=FAKE + 2) == 1 and call(f32=0, logits=FAKE + 1) == 1
    for name in ("u", "t", "k", "p", "m", "tok", "lp"):
        assert call(**{name: FAKE + 2}) == 1, name
    assert call(f32=2) == 1 and call(ld=999) == 1 and call(B=-1) == 1 and call(V=0) == 1
    assert call(V=(1 << 22) + 1, ld=1 << 23) == 2 and call(B=65536) == 2
    assert call(B=65535, V=1 << 22, ld=1 << 22) == 2 and size(65535, 1 << 22) == 0  # more threads than a launch's
    assert call(scratch=None) == 3 and call(nbytes=64) == 3 and call(scratch=FAKE + 128) == 3
    assert call(B=0) == 0


def test_sampling_binding_refuses_what_is_not_on_the_device():
    with pytest.raises(ValueError):
        ge.engram_sample(torch.zeros(4, 16), torch.zeros(4))
    with pytest.raises(TypeError):
        ge.engram_sample([1.0], torch.zeros(4))


def test_outputs_that_overlap_inputs_are_refused():
    lib = ge.load()
    at = [(i + 1) << 32 for i in range(9)]  # far apart: refused for the one overlap that each call has
    table, ids, scratch = at[0], at[1], at[2]

    def embed(out, o32=0, streams=2):  # out: 4 * 2 * 64 values; the table 100 * 64 of bf16
        return lib.engram_embed(table, 0, 100, 64, ids, 4, 1.0, streams, out, o32, None, None)
    assert embed(table) == 1 and embed(table + 100 * 128 - 16) == 1 and embed(table - 1024 + 16) == 1
    assert embed(table - 2048 + 16, o32=1) == 1 and embed(ids) == 1

    def grad(dt, n=4, t32=0):
        return lib.engram_embed_grad(table, 0, ids, n, 2, 100, 64, 1.0, -1, 0, dt, t32, scratch, 1 << 30, None, None)
    assert grad(table) == 1 and grad(table + 4 * 256 - 16) == 1 and grad(table - 100 * 128 + 16) == 1
    assert grad(table - 100 * 256 + 16, t32=1) == 1 and grad(ids) == 1

    names = ("u", "t", "k", "p", "m", "tok", "lp")
    places = dict(zip(names, at[2:]))

    def sample(**where):
        p = {**places, **where}
        return lib.engram_sample(at[0], 0, 1000, p["u"], p["t"], p["k"], p["p"], p["m"], 3, 900, p["tok"], p["lp"],
                                 at[1], 1 << 30, None, None)
    for out in ("tok", "lp"):
        for name in names:
            if name != out:
                assert sample(**{out: places[name] + 8}) == 1 and sample(**{out: places[name] - 8}) == 1, (out, name)
        assert sample(**{out: at[0] + 2 * 2900 - 4}) == 1 and sample(**{out: at[0] - 8}) == 1, out


def test_scratch_that_overlaps_anything_is_refused():
    """Scratch is written and read by every launch of a call, err by some; each call here has one overlap, of
    its first or its last bytes."""
    lib = ge.load()
    at = [(i + 1) << 34 for i in range(10)]
    n, rows, dim, streams = 100, 1000, 64, 2
    need = ge.engram_embed_grad_scratch_size(n, rows, dim)
    held = {"dout": n * streams * dim * 2, "ids": n * 4, "dt": rows * dim * 4}
    places = dict(zip(held, at))

    def grad(scratch, err=None, **where):
        p = {**places, **where}
        return lib.engram_embed_grad(p["dout"], 0, p["ids"], n, streams, rows, dim, 1.0, -1, 0, p["dt"], 1, scratch,
                                     1 << 30, err, None)
    for name, size in held.items():
        first = at[9] + (need - 4 if name == "ids" else need - 16)
        assert grad(at[9], **{name: first}) == 1, name
        assert grad(places[name] + size // 256 * 256 - (0 if size % 256 else 256)) == 1, name
        for err in (places[name], places[name] + size - 4):
            assert grad(at[9], err) == 1, name
    assert grad(at[9], at[9]) == 1 and grad(at[9], at[9] + need - 4) == 1

    B, V, ld = 3, 900, 1000
    need = ge.engram_sample_scratch_size(B, V)
    held = {"logits": ((B - 1) * ld + V) * 2, **{name: B * 4 for name in ("u", "t", "k", "p", "m", "tok", "lp")}}
    places = dict(zip(held, at))

    def sample(scratch, err=None, **where):
        p = {**places, **where}
        return lib.engram_sample(p["logits"], 0, ld, p["u"], p["t"], p["k"], p["p"], p["m"], B, V, p["tok"], p["lp"],
                                 scratch, 1 << 30, err, None)
    for name, size in held.items():
        assert sample(at[9], **{name: at[9] + need - 4}) == 1, name
        assert sample(places[name]) == 1, name
        for err in (places[name], places[name] + size - 4):
            assert sample(at[9], err) == 1, name
    assert sample(at[9], at[9]) == 1 and sample(at[9], at[9] + need - 4) == 1

    def embed(err):
        return lib.engram_embed(at[0], 0, rows, dim, at[1], n, 1.0, streams, at[2], 0, err, None)
    for err in (at[0], at[0] + rows * dim * 2 - 4, at[1], at[1] + n * 4 - 4, at[2], at[2] + n * streams * dim * 2 - 4):
        assert embed(err) == 1
