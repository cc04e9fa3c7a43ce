"""The calls around the layer in serving (adapters, norm to 8 bits, beam
selection, state reordering) without a GPU: sizes and refusals.  Every call
here fails its checks on the host, or has no work, and launches nothing."""
import ctypes as C

import pytest
import torch

import gram_memory_layer_amd as ge

FAKE = 1 << 20  # never dereferenced


def geom():
    return ge.Geometry.make(dim=5120, hc_mult=4, max_ngram_size=3, n_heads=12, head_dim=64,
                            num_embeddings=25160950, vocab=129280)


def c_adapters(down=FAKE, up=FAKE, scale=None, n=4, rank=16):
    return ge._CAdapters(down, up, scale, n, rank)


def test_adapters_host_checks():
    lib, g = ge.load(), geom()
    ok = c_adapters()
    size = lambda ad, M: lib.engram_wkv_adapters_scratch_size(C.byref(g), C.byref(ad), M)  # noqa: E731
    # ranks in whole 16s, a pair of bf16 each, then 8 bytes for each of the tiles' rows (whole 256s)
    assert size(ok, 64) == 64 * 16 * 4 + 256 * 8
    assert size(c_adapters(rank=24), 300) == 300 * 32 * 4 + 512 * 8
    assert size(ok, 0) == 0 and size(ok, -1) == 0

    def call(ad=ok, a=FAKE, w=FAKE, ids=FAKE, M=8, kv=FAKE, scratch=FAKE, nbytes=1 << 30):
        return lib.engram_wkv_adapters(C.byref(g), C.byref(ad) if ad else None, a, w, ids, M, kv,
                                       scratch, nbytes, None, None)
    assert call(ad=None) == 1
    assert call(ad=c_adapters(down=None)) == 1 and call(ad=c_adapters(up=None)) == 1
    assert call(ad=c_adapters(down=FAKE + 8)) == 1 and call(ad=c_adapters(up=FAKE + 2)) == 1
    assert call(ad=c_adapters(scale=FAKE + 2)) == 1
    for kw in (dict(n=0), dict(n=65537), dict(rank=0), dict(rank=12), dict(rank=136)):
        assert call(ad=c_adapters(**kw)) == 2, kw
        assert size(c_adapters(**kw), 8) == 0
    assert call(a=None) == 1 and call(w=None) == 1 and call(ids=None) == 1 and call(kv=None) == 1
    assert call(a=FAKE + 8) == 1 and call(kv=FAKE + 8) == 1 and call(ids=FAKE + 1) == 1
    assert call(M=-1) == 1
    assert call(scratch=None) == 3 and call(nbytes=255) == 3 and call(scratch=FAKE + 64) == 3
    assert call(M=0) == 0
    bad = geom()
    bad.head_dim = 40
    assert lib.engram_wkv_adapters(C.byref(bad), C.byref(ok), FAKE, FAKE, FAKE, 8, FAKE, FAKE,
                                   1 << 30, None, None) == 2


def test_forward_adapted_host_checks():
    lib, g, ok = ge.load(), geom(), c_adapters()
    ht = ge.HashTables(FAKE, FAKE, FAKE, FAKE)
    need = lib.engram_forward_adapted_workspace_size(C.byref(g), C.byref(ok), 8)
    assert need == ge.engram_forward_workspace_size(g, 8) + 8 * 16 * 4 + 256 * 8
    assert lib.engram_forward_adapted_workspace_size(C.byref(g), C.byref(c_adapters(n=0)), 8) == 0

    def call(ad=ok, ids=FAKE, aid=FAKE, B=2, T=4, ws=FAKE, nbytes=need):
        return lib.engram_forward_adapted(C.byref(g), C.byref(ht), C.byref(ad), FAKE, FAKE, FAKE,
                                          FAKE, FAKE, None, FAKE, ids, aid, None, B, T, FAKE, None,
                                          ws, nbytes, None, None)
    assert call(ids=None) == 1 and call(aid=None) == 1 and call(aid=FAKE + 2) == 1
    assert call(B=-1) == 1 and call(ad=c_adapters(rank=9)) == 2
    assert call(ws=None) == 3 and call(nbytes=need - 1) == 3 and call(ws=FAKE + 16) == 3
    assert call(B=0) == 0


def test_norm_quant_host_checks():
    lib = ge.load()

    def call(x=FAKE, res=None, w=None, rows=4, dim=64, eps=1e-6, fmt=0, total=None, codes=FAKE,
             scales=FAKE):
        return lib.engram_norm_quant(x, res, w, rows, dim, eps, fmt, total, codes, scales, None)
    assert call(x=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1
    assert call(x=FAKE + 2) == 1 and call(res=FAKE + 8) == 1 and call(w=FAKE + 8) == 1
    assert call(total=FAKE + 8) == 1 and call(codes=FAKE + 4) == 1
    assert call(fmt=1, scales=FAKE + 2) == 1
    assert call(fmt=-1) == 1 and call(fmt=3) == 1
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(eps=float("nan")) == 1 and call(eps=-1.0) == 1 and call(eps=float("inf")) == 1
    for dim in (0, 4, 12, 32776):
        assert call(dim=dim) == 2, dim
    assert call(rows=0) == 0


def test_beam_select_host_checks():
    lib = ge.load()
    size = ge.engram_beam_select_scratch_size
    assert size(2, 4, 1000) > 0 and size(0, 4, 1000) == 0 and size(2, 33, 1000) == 0

    def call(logits=FAKE, f32=1, ld=1000, scores=FAKE, fin=None, B=2, W=4, V=1000, eos=1, pad=0,
             tok=FAKE, par=FAKE, ns=FAKE, nf=None, scratch=FAKE, nbytes=1 << 40):
        return lib.engram_beam_select(logits, f32, ld, scores, fin, B, W, V, eos, pad, tok, par,
                                      ns, nf, scratch, nbytes, None, None)
    assert call(logits=None) == 1 and call(scores=None) == 1 and call(tok=None) == 1
    assert call(par=None) == 1 and call(ns=None) == 1
    assert call(logits=FAKE + 2) == 1 and call(f32=0, logits=FAKE + 1) == 1
    assert call(scores=FAKE + 1) == 1
    assert call(f32=2) == 1 and call(ld=999) == 1
    assert call(pad=-1) == 1 and call(pad=1000) == 1 and call(eos=-2) == 1
    assert call(B=-1) == 1 and call(W=0) == 1 and call(V=0) == 1
    assert call(W=33) == 2 and call(V=3, ld=3) == 2 and call(B=16384) == 2
    assert call(V=(1 << 30) + 1, ld=1 << 31) == 2
    assert call(W=4, V=1 << 29, ld=1 << 31) == 2
    assert call(scratch=None) == 3 and call(nbytes=64) == 3 and call(scratch=FAKE + 128) == 3
    assert call(B=0) == 0


def test_beam_reorder_host_checks():
    lib = ge.load()

    def call(ptrs=(FAKE,), size=(8,), n=None, parents=FAKE, B=2, W=4):
        n = len(ptrs) if n is None else n
        p = (C.c_void_p * max(len(ptrs), 1))(*ptrs)
        s = (C.c_int64 * max(len(size), 1))(*size)
        return lib.engram_beam_reorder(p, s, n, parents, B, W, None, None)
    assert lib.engram_beam_reorder(None, None, 1, FAKE, 2, 4, None, None) == 1
    assert call(n=0) == 1 and call(ptrs=(FAKE,) * 33, size=(8,) * 33) == 1
    assert call(size=(6,)) == 1 and call(size=(0,)) == 1 and call(size=(1 << 37,)) == 2
    assert call(ptrs=(None,)) == 1 and call(ptrs=(FAKE + 2,)) == 1
    assert call(parents=None) == 1 and call(parents=FAKE + 2) == 1
    assert call(B=-1) == 1 and call(W=0) == 1 and call(W=33) == 2 and call(B=65536) == 2
    # 2 * 4 rows of 8 bytes: 64 bytes; the second state starts inside the first
    assert call(ptrs=(FAKE, FAKE + 60), size=(8, 8)) == 1
    assert call(ptrs=(FAKE + 60, FAKE), size=(8, 8)) == 1
    assert call(ptrs=(FAKE, FAKE), size=(8, 8)) == 1
    assert call(B=0) == 0


def test_binding_refuses_what_is_not_on_the_device():
    g = geom()
    with pytest.raises(ValueError):
        ge.Adapters(torch.zeros(2, 8, 1536, dtype=torch.bfloat16),
                    torch.zeros(2, 25600, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ge.engram_norm_quant(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ge.engram_norm_quant(torch.zeros(4, 64, dtype=torch.bfloat16), scale_format="e8m0")
    with pytest.raises(ValueError):
        ge.engram_beam_select(torch.zeros(4, 64), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        ge.engram_beam_reorder([torch.zeros(4, 2)], torch.zeros(1, 4, dtype=torch.int32))
    layer = ge.EngramLayer.__new__(ge.EngramLayer)
    with pytest.raises(ValueError):  # ids that no adapters go with
        layer.forward(torch.zeros(1, 1, 4, 5120, dtype=torch.bfloat16), torch.zeros(1, 1),
                      adapter_ids=torch.zeros(1, dtype=torch.int32))
    assert g.K == 1536
